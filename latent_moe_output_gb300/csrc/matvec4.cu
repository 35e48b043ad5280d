// latent_tail_expert_matvec4: products of expert-sorted rows with 4-bit weights
// that carry one scale per group of G columns.
//
//   out[r,m] = sum_c x[r,c] * (q[e,m,c] - 8) * s[e,m,c/G]
//
// First form: one warp per output element.
#include "block_launch.h"
#include "rows.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    matvec4_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ packed,
                   const uint16_t* __restrict__ scales, const int32_t* __restrict__ offsets,
                   uint16_t* __restrict__ out, int N, int E, int M, int C, int G) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t elements = static_cast<int64_t>(N) * M;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       id < elements; id += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
    const int r = static_cast<int>(id / M), m = static_cast<int>(id % M);
    int e = 0;
    if (offsets != nullptr) {  // first expert whose rows end after r
      int hi = E;
      while (e < hi) {
        const int mid = (e + hi) / 2;
        if (offsets[mid + 1] > r)
          hi = mid;
        else
          e = mid + 1;
      }
    }
    float sum = 0.f;
    if (e < E) {
      const size_t row = static_cast<size_t>(e) * M + m;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(packed + row * (C / 2));
      for (int w = lane; w < C / 8; w += 32) {  // eight weights
        const uint32_t bits = q[w];
        float a[8];
        unpack8(ld_stream_v4(x + static_cast<size_t>(r) * C + w * 8), a);
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          part = fmaf(a[i], static_cast<float>(static_cast<int>((bits >> (4 * i)) & 15u) - 8), part);
        const float s = bf16_lo(scales[row * (C / G) + w * 8 / G]);
        sum = fmaf(part, s, sum);
      }
    }
    sum = warp_sum_f(sum);
    if (lane == 0) out[static_cast<size_t>(r) * M + m] =
        static_cast<uint16_t>(pack_bf16x2(sum, 0.f) & 0xffffu);
  }
}

}  // namespace

cudaError_t setup_matvec4(const DeviceInfo&) { return cudaSuccess; }

cudaError_t launch_matvec4(const Matvec4Args& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t ctas = (static_cast<int64_t>(a.N) * a.M + 7) / 8;
  return launch_dependent(matvec4_kernel,
                          dim3(static_cast<unsigned>(std::min<int64_t>(ctas, dev.num_sms * 8))),
                          dim3(kThreads), 0, stream, a.x, a.packed, a.scales, a.offsets, a.out,
                          a.N, a.E, a.M, a.C, a.G);
}

}  // namespace lt
