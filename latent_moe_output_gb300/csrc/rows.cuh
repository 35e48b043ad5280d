// Small device helpers shared by the row-wise kernels: 8-element vectors in
// FP32, warp and thread-group sums, programmatic-dependent launches.
#pragma once

#include "ptx.cuh"

#include <utility>

namespace lt {

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 16-byte load of data that this kernel may overwrite afterwards (an in-place
// residual), so not through the read-only path.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&a)[8]) {
  a[0] = bf16_lo(v.x);
  a[1] = bf16_hi(v.x);
  a[2] = bf16_lo(v.y);
  a[3] = bf16_hi(v.y);
  a[4] = bf16_lo(v.z);
  a[5] = bf16_hi(v.z);
  a[6] = bf16_lo(v.w);
  a[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

// Two FP32 values in a register pair: one packed instruction does both, with the
// same rounding as the scalar one.
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ void split(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float lo, hi;
  split(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& v, f32x2 (&a)[4]) {
  a[0] = pair(bf16_lo(v.x), bf16_hi(v.x));
  a[1] = pair(bf16_lo(v.y), bf16_hi(v.y));
  a[2] = pair(bf16_lo(v.z), bf16_hi(v.z));
  a[3] = pair(bf16_lo(v.w), bf16_hi(v.w));
}

__device__ __forceinline__ uint32_t pack_bf16x2(f32x2 v) {
  float lo, hi;
  split(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const f32x2 (&a)[4]) {
  return make_uint4(pack_bf16x2(a[0]), pack_bf16x2(a[1]), pack_bf16x2(a[2]), pack_bf16x2(a[3]));
}

// One kernel launch as a programmatic dependent of the work before it on the
// stream: the kernel may start early and must call pdl_wait() before it reads
// or writes memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent_clusters(unsigned cluster, void (*kernel)(KArgs...), dim3 grid,
                                      dim3 block, size_t smem, cudaStream_t stream,
                                      Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, Args&&... args) {
  return launch_dependent_clusters(1, kernel, grid, block, smem, stream,
                                   std::forward<Args>(args)...);
}

}  // namespace lt
