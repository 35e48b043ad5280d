// latent_tail_combine and its gradient: the experts' rows summed back to their
// tokens with the router's weights.
//
//   out[t]     = sum_k w[t,k] * rows[position[t,k]]        (k ascending, FP32)
//   grad_rows[position[t,k]] = w[t,k] * grad_out[t]
//   grad_w[t,k] = <grad_out[t], rows[position[t,k]]>
//
// Both read and write every row once, so memory bounds them.
#include "block_launch.h"
#include "rows.cuh"

namespace lt {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // rows requested before the first is used

// One thread per 16-byte piece of out.
__global__ void __launch_bounds__(kThreads)
    combine_kernel(const uint16_t* __restrict__ rows, const int32_t* __restrict__ position,
                   const float* __restrict__ weights, uint16_t* __restrict__ out, int T, int K,
                   int nch) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int t0 = static_cast<int>(base / nch);
  const int rem = static_cast<int>(base - static_cast<int64_t>(t0) * nch) + threadIdx.x;
  const int t = t0 + rem / nch, c = rem % nch;
  if (t >= T) return;
  const int n = T * K;
  const size_t at = static_cast<size_t>(t) * K;
  const uint4* src = reinterpret_cast<const uint4*>(rows) + c;
  float acc[8] = {};
  for (int k0 = 0; k0 < K; k0 += kAhead) {
    uint4 v[kAhead];
    float w[kAhead];
    bool on[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j;
      const int p = k < K ? position[at + k] : -1;
      on[j] = p >= 0 && p < n;
      v[j] = on[j] ? ld_stream_v4(src + static_cast<size_t>(p) * nch) : make_uint4(0, 0, 0, 0);
      w[j] = on[j] && weights != nullptr ? weights[at + k] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!on[j]) continue;
      float a[8];
      unpack8(v[j], a);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], a[i], acc[i]);
    }
  }
  reinterpret_cast<uint4*>(out)[static_cast<size_t>(t) * nch + c] = pack8(acc);
}

// A group of `tpt` threads (a power of two, 8 to 256) per token; each thread owns
// every tpt-th 16-byte piece of the token's row.
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const uint16_t* __restrict__ grad_out,
                            const uint16_t* __restrict__ rows,
                            const int32_t* __restrict__ position,
                            const float* __restrict__ weights, uint16_t* __restrict__ grad_rows,
                            float* __restrict__ grad_weights, int T, int K, int nch, int tpt) {
  __shared__ float s_dot[kThreads / 32][kAhead];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & (tpt - 1);
  const int t = blockIdx.x * (kThreads / tpt) + threadIdx.x / tpt;
  const bool live = t < T;
  const int n = T * K;
  const size_t at = static_cast<size_t>(t) * K;
  const uint4* g4 = reinterpret_cast<const uint4*>(grad_out) + static_cast<size_t>(t) * nch;
  const uint4* r4 = reinterpret_cast<const uint4*>(rows);
  uint4* d4 = reinterpret_cast<uint4*>(grad_rows);
  for (int k0 = 0; k0 < K; k0 += kAhead) {
    int place[kAhead];  // row of grad_rows, or -1
    float w[kAhead];
    bool on[kAhead];
    float dot[kAhead] = {};
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j;
      const bool have = live && k < K;
      const int p = have ? position[at + k] : -1;
      const int row = p >= 0 ? p : ~p;
      on[j] = have && p >= 0 && p < n;
      place[j] = have && row < n ? row : -1;
      w[j] = !on[j] ? 0.f : weights != nullptr ? weights[at + k] : 1.f;
    }
    if (live) {
      for (int c = lane; c < nch; c += tpt) {
        const uint4 gv = ld_stream_v4(g4 + c);
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          v[j] = on[j] && grad_weights != nullptr
                     ? ld_stream_v4(r4 + static_cast<size_t>(place[j]) * nch + c)
                     : make_uint4(0, 0, 0, 0);
        float g[8];
        unpack8(gv, g);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (place[j] < 0) continue;
          float a[8];
          if (on[j]) {
            unpack8(v[j], a);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], a[i], dot[j]);
          }
          // A choice without an expert gets zeros even where grad_out is not finite.
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = on[j] ? w[j] * g[i] : 0.f;
          d4[static_cast<size_t>(place[j]) * nch + c] = pack8(a);
        }
      }
    }
    if (grad_weights == nullptr) continue;
    const int span = tpt < 32 ? tpt : 32;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      for (int o = span / 2; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    if (tpt > 32) {  // the warps of a token add up in warp order
      const int warp = threadIdx.x >> 5;
      __syncthreads();
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < kAhead; ++j) s_dot[warp][j] = dot[j];
      __syncthreads();
      const int j = lane;
      if (live && j < kAhead && k0 + j < K) {
        const int w0 = threadIdx.x / tpt * (tpt / 32);
        float sum = 0.f;
        for (int i = 0; i < tpt / 32; ++i) sum += s_dot[w0 + i][j];
        grad_weights[at + k0 + j] = sum;
      }
    } else if (live && lane == 0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (k0 + j < K) grad_weights[at + k0 + j] = dot[j];
    }
  }
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, const DeviceInfo&, cudaStream_t stream) {
  const int nch = a.L / 8;
  const int64_t pieces = static_cast<int64_t>(a.T) * nch;
  return launch_dependent(combine_kernel,
                          dim3(static_cast<unsigned>((pieces + kThreads - 1) / kThreads)),
                          dim3(kThreads), 0, stream, a.rows, a.position, a.weights, a.out, a.T,
                          a.K, nch);
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, const DeviceInfo&,
                                    cudaStream_t stream) {
  const int nch = a.L / 8;
  int tpt = 8;
  while (tpt < nch && tpt < kThreads) tpt *= 2;
  const int per_cta = kThreads / tpt;
  return launch_dependent(combine_backward_kernel, dim3((a.T + per_cta - 1) / per_cta),
                          dim3(kThreads), 0, stream, a.grad_out, a.rows, a.position, a.weights,
                          a.grad_rows, a.grad_weights, a.T, a.K, nch, tpt);
}

}  // namespace lt
