// latent_tail_combine and its gradient: the experts' rows summed back to their
// tokens with the router's weights.
//
//   out[t]     = sum_k w[t,k] * rows[position[t,k]]        (k ascending, FP32)
//   grad_rows[position[t,k]] = w[t,k] * grad_out[t]
//   grad_w[t,k] = <grad_out[t], rows[position[t,k]]>
//
// Both read and write every row once, so memory bounds them. Measured at K = 8,
// L = 2048 (GB300, calls back to back): 8192 tokens with a quarter of the choices not
// routed 37.1 us = 6.3 TB/s, 93 % of the measured copy rate; the gradient of 8192 tokens
// 86 us = 6.6 TB/s, 97 %; 16 tokens 1.9 us.
#include "block_launch.h"
#include "rows.cuh"

namespace lt {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // rows requested before the first is used
// Threads of the forward kernel: T = 8192, a quarter not routed, 37.1 us with 128, 38.1
// with 256, 40.4 with 512; T = 16 1.9, 2.1 and 2.5.
constexpr int kForwardThreads = 128;

// One thread per 16-byte piece of out.
__global__ void __launch_bounds__(kForwardThreads)
    combine_kernel(const uint16_t* __restrict__ rows, const int32_t* __restrict__ position,
                   const float* __restrict__ weights, uint16_t* __restrict__ out, int T, int K,
                   int nch) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kForwardThreads;
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
  st_stream_v4(reinterpret_cast<uint4*>(out) + static_cast<size_t>(t) * nch + c, pack8(acc));
}

// A group of kTpt threads per token; each thread owns every kTpt-th 16-byte piece of
// the token's row. Lane j of the group holds choice k0 + j. The rows are requested
// first, the gradients of the rows (which do not need them) written meanwhile, the
// products with the rows summed last; four CTAs per SM overlap the three steps. At
// T = 8192, K = 8, L = 2048: 85 us with streaming stores (the rows are not read again
// here), 88 with plain ones, 92 with three CTAs per SM, 113 with two.
template <int kTpt>
__global__ void __launch_bounds__(kThreads, 4)
    combine_backward_kernel(const uint16_t* __restrict__ grad_out,
                            const uint16_t* __restrict__ rows,
                            const int32_t* __restrict__ position,
                            const float* __restrict__ weights, uint16_t* __restrict__ grad_rows,
                            float* __restrict__ grad_weights, int T, int K, int nch) {
  constexpr int kSpan = kTpt < 32 ? kTpt : 32;  // lanes of one token in a warp
  __shared__ float s_dot[kThreads / 32][kAhead];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kTpt, wlane = threadIdx.x & 31, first = wlane & ~(kSpan - 1);
  const int t = blockIdx.x * (kThreads / kTpt) + threadIdx.x / kTpt;
  const bool live = t < T;
  const int n = T * K;
  const size_t at = static_cast<size_t>(t) * K;
  const uint4* g4 = reinterpret_cast<const uint4*>(grad_out) + static_cast<size_t>(t) * nch;
  const uint4* r4 = reinterpret_cast<const uint4*>(rows);
  uint4* d4 = reinterpret_cast<uint4*>(grad_rows);
  const bool dots = grad_weights != nullptr;
  for (int k0 = 0; k0 < K; k0 += kAhead) {
    int mine = n;  // position of choice k0 + j in lane j; n: none
    float my_w = 0.f;
    const int j0 = wlane - first;
    if (live && j0 < kAhead && k0 + j0 < K) {
      mine = position[at + k0 + j0];
      if (mine >= 0 && mine < n) my_w = weights != nullptr ? weights[at + k0 + j0] : 1.f;
    }
    float dot[kAhead] = {};
    const int chunks = (nch + kTpt - 1) / kTpt;
    for (int i = 0; i < chunks; ++i) {
      const int c = lane + i * kTpt;
      const bool have = live && c < nch;
      uint4 v[kAhead], gv = make_uint4(0, 0, 0, 0);
      if (have) gv = ld_stream_v4(g4 + c);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int p = __shfl_sync(0xffffffffu, mine, first + j);
        v[j] = make_uint4(0, 0, 0, 0);
        if (have && dots && p >= 0 && p < n) v[j] = ld_stream_v4(r4 + static_cast<size_t>(p) * nch + c);
      }
      f32x2 g[4];
      unpack8(gv, g);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int p = __shfl_sync(0xffffffffu, mine, first + j);
        const f32x2 w = both(__shfl_sync(0xffffffffu, my_w, first + j));
        const int row = p >= 0 ? p : ~p;
        f32x2 d[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = mul2(w, g[q]);
        // A choice without an expert gets zeros even where grad_out is not finite.
        if (have && row < n)
          st_stream_v4(d4 + static_cast<size_t>(row) * nch + c,
                       p >= 0 ? pack8(d) : make_uint4(0, 0, 0, 0));
      }
      if (dots) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          f32x2 a[4], q = both(0.f);
          unpack8(v[j], a);
#pragma unroll
          for (int u = 0; u < 4; ++u) q = fma2(g[u], a[u], q);
          const int p = __shfl_sync(0xffffffffu, mine, first + j);
          if (p >= 0 && p < n) dot[j] += sum2(q);  // (zeros times an infinity are not added)
        }
      }
    }
    if (!dots) continue;
    if constexpr (kTpt < 32) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int o = kSpan / 2; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (live && lane == 0)
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k0 + j < K) grad_weights[at + k0 + j] = dot[j];
    } else {
      // Halving exchanges leave lanes 4 j .. 4 j + 3 with parts of dot[j].
#pragma unroll
      for (int m = kAhead / 2, o = 16; m > 0; m /= 2, o /= 2) {
        const bool up = wlane & o;
#pragma unroll
        for (int j = 0; j < m; ++j)
          dot[j] = (up ? dot[m + j] : dot[j]) +
                   __shfl_xor_sync(0xffffffffu, up ? dot[j] : dot[m + j], o);
      }
      float sum = dot[0];
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      const int j = wlane >> 2;
      if constexpr (kTpt == 32) {
        if (live && (wlane & 3) == 0 && k0 + j < K) grad_weights[at + k0 + j] = sum;
      } else {  // the warps of a token add up in warp order
        const int warp = threadIdx.x >> 5;
        if (k0 > 0) __syncthreads();
        if ((wlane & 3) == 0) s_dot[warp][j] = sum;
        __syncthreads();
        if (live && lane < kAhead && k0 + lane < K) {
          sum = 0.f;
#pragma unroll
          for (int i = 0; i < kTpt / 32; ++i) sum += s_dot[threadIdx.x / kTpt * (kTpt / 32) + i][lane];
          grad_weights[at + k0 + lane] = sum;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, const DeviceInfo&, cudaStream_t stream) {
  const int nch = a.L / 8;
  const int64_t pieces = static_cast<int64_t>(a.T) * nch;
  return launch_dependent(combine_kernel,
                          dim3(static_cast<unsigned>((pieces + kForwardThreads - 1) /
                                                     kForwardThreads)),
                          dim3(kForwardThreads), 0, stream, a.rows, a.position, a.weights, a.out, a.T,
                          a.K, nch);
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, const DeviceInfo&,
                                    cudaStream_t stream) {
  const int nch = a.L / 8;
  int tpt = 8;
  while (tpt < nch && tpt < kThreads) tpt *= 2;
  auto* k = tpt == 8     ? combine_backward_kernel<8>
            : tpt == 16  ? combine_backward_kernel<16>
            : tpt == 32  ? combine_backward_kernel<32>
            : tpt == 64  ? combine_backward_kernel<64>
            : tpt == 128 ? combine_backward_kernel<128>
                         : combine_backward_kernel<256>;
  const int per_cta = kThreads / tpt;
  return launch_dependent(k, dim3((a.T + per_cta - 1) / per_cta), dim3(kThreads), 0, stream,
                          a.grad_out, a.rows, a.position, a.weights, a.grad_rows, a.grad_weights,
                          a.T, a.K, nch);
}

}  // namespace lt
