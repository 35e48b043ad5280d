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
// Threads of the forward kernel: T = 8192, a quarter not routed, 37.1 us with 128, 38.1
// with 256, 40.4 with 512; T = 16 1.9, 2.1 and 2.5.
constexpr int kForwardThreads = 128;

// One thread per kPieces 16-byte pieces of out, kForwardThreads apart, kRowsAhead choices
// at a time.
template <int kRowsAhead, int kPieces>
__global__ void __launch_bounds__(kForwardThreads)
    combine_kernel(const uint16_t* __restrict__ rows, const int32_t* __restrict__ position,
                   const float* __restrict__ weights, uint16_t* __restrict__ out, int T, int K,
                   int nch) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kForwardThreads * kPieces);
  const int t0 = static_cast<int>(base / nch);
  const int rem0 = static_cast<int>(base - static_cast<int64_t>(t0) * nch) + threadIdx.x;
  const int n = T * K;
  const uint4* src = reinterpret_cast<const uint4*>(rows);
  int t[kPieces], c[kPieces];
  float acc[kPieces][8] = {};
#pragma unroll
  for (int e = 0; e < kPieces; ++e) {
    const int rem = rem0 + e * kForwardThreads;
    t[e] = t0 + rem / nch;
    c[e] = rem % nch;
  }
  if (kPieces == 1 && t[0] >= T) return;
  for (int k0 = 0; k0 < K; k0 += kRowsAhead) {
    uint4 v[kPieces][kRowsAhead];
    float w[kPieces][kRowsAhead];
    bool on[kPieces][kRowsAhead];
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        const int k = k0 + j;
        const size_t at = static_cast<size_t>(t[e]) * K + k;
        const int p = (kPieces == 1 || t[e] < T) && k < K ? position[at] : -1;
        on[e][j] = p >= 0 && p < n;
        v[e][j] = on[e][j] ? ld_stream_v4(src + static_cast<size_t>(p) * nch + c[e])
                           : make_uint4(0, 0, 0, 0);
        w[e][j] = on[e][j] && weights != nullptr ? weights[at] : 1.f;
      }
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        if (!on[e][j]) continue;
        float a[8];
        unpack8(v[e][j], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[e][i] = fmaf(w[e][j], a[i], acc[e][i]);
      }
  }
#pragma unroll
  for (int e = 0; e < kPieces; ++e)
    if (kPieces == 1 || t[e] < T)
      st_stream_v4(reinterpret_cast<uint4*>(out) + static_cast<size_t>(t[e]) * nch + c[e],
                   pack8(acc[e]));
}

// Gradient: 16-byte pieces per thread in flight. With few choices per token one piece
// leaves the memory idle (us with one row of eight slots used by K, and with two pieces
// of K rows rounded up to 2 or 4: T = 16384, K = 1, L = 512 21.6 and 10.1; T = 2048, K = 2,
// L = 4096 20.6 and 14.4; T = 8192, K = 3, L = 1448 42.9 and 31.0). Within the 64
// registers of four CTAs per SM the kernels of four slots spill 52-92 bytes, those of
// eight 24-44; four pieces per thread spill 184 to 508.
constexpr int pieces_ahead(int rows_ahead) { return rows_ahead == 8 ? 1 : 2; }

// A group of kTpt threads per token; each thread owns every kTpt-th 16-byte piece of
// the token's row. Lane j of the group holds choice k0 + j. The rows are requested
// first, the gradients of the rows (which do not need them) written meanwhile, the
// products with the rows summed last; four CTAs per SM overlap the three steps. At
// T = 8192, K = 8, L = 2048: 85 us with streaming stores (the rows are not read again
// here), 88 with plain ones, 92 with three CTAs per SM, 113 with two.
template <int kTpt, int kAhead>
__global__ void __launch_bounds__(kThreads, 4)
    combine_backward_kernel(const uint16_t* __restrict__ grad_out,
                            const uint16_t* __restrict__ rows,
                            const int32_t* __restrict__ position,
                            const float* __restrict__ weights, uint16_t* __restrict__ grad_rows,
                            float* __restrict__ grad_weights, int T, int K, int nch) {
  constexpr int kUnroll = pieces_ahead(kAhead);
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
    for (int i = 0; i < chunks; i += kUnroll) {
      uint4 v[kUnroll][kAhead], gv[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = lane + (i + u) * kTpt;
        const bool have = live && c < nch;
        gv[u] = have ? ld_stream_v4(g4 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int p = __shfl_sync(0xffffffffu, mine, first + j);
          v[u][j] = make_uint4(0, 0, 0, 0);
          if (have && dots && p >= 0 && p < n)
            v[u][j] = ld_stream_v4(r4 + static_cast<size_t>(p) * nch + c);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = lane + (i + u) * kTpt;
        const bool have = live && c < nch;
        f32x2 g[4];
        unpack8(gv[u], g);
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
      }
      if (dots) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          f32x2 g[4];
          unpack8(gv[u], g);
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            f32x2 a[4], q = both(0.f);
            unpack8(v[u][j], a);
#pragma unroll
            for (int m = 0; m < 4; ++m) q = fma2(g[m], a[m], q);
            const int p = __shfl_sync(0xffffffffu, mine, first + j);
            if (p >= 0 && p < n) dot[j] += sum2(q);  // (zeros times an infinity are not added)
          }
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
      // Halving exchanges leave each kLanes lanes with parts of one dot[j].
      constexpr int kLanes = 32 / kAhead;
#pragma unroll
      for (int m = kAhead / 2, o = 16; m > 0; m /= 2, o /= 2) {
        const bool up = wlane & o;
#pragma unroll
        for (int j = 0; j < m; ++j)
          dot[j] = (up ? dot[m + j] : dot[j]) +
                   __shfl_xor_sync(0xffffffffu, up ? dot[j] : dot[m + j], o);
      }
      float sum = dot[0];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int j = wlane / kLanes;
      if constexpr (kTpt == 32) {
        if (live && wlane % kLanes == 0 && k0 + j < K) grad_weights[at + k0 + j] = sum;
      } else {  // the warps of a token add up in warp order
        const int warp = threadIdx.x >> 5;
        if (k0 > 0) __syncthreads();
        if (wlane % kLanes == 0) s_dot[warp][j] = sum;
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

template <int kAhead>
auto backward_kernel(int tpt) {
  return tpt == 8     ? combine_backward_kernel<8, kAhead>
         : tpt == 16  ? combine_backward_kernel<16, kAhead>
         : tpt == 32  ? combine_backward_kernel<32, kAhead>
         : tpt == 64  ? combine_backward_kernel<64, kAhead>
         : tpt == 128 ? combine_backward_kernel<128, kAhead>
                      : combine_backward_kernel<256, kAhead>;
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int nch = a.L / 8;
  const int64_t pieces = static_cast<int64_t>(a.T) * nch;
  // Few choices per token: more pieces per thread, to have as many rows in flight (us with
  // one piece and with more: T = 16384, K = 1, L = 512 14.5 and 6.9; T = 2048, K = 2, L =
  // 4096 14.7 and 8.3; T = 8192, K = 4, L = 1024 16.9 and 13.8; T = 256, K = 4, L = 2048
  // 3.0 and 2.7), unless they would not fill one CTA per SM.
  int per = a.K == 1 ? 4 : a.K <= 4 ? 2 : 1;
  if (pieces < static_cast<int64_t>(dev.num_sms) * kForwardThreads * per) per = 1;
  const int64_t per_cta = static_cast<int64_t>(kForwardThreads) * per;
  return launch_dependent(per == 1      ? combine_kernel<8, 1>
                          : a.K == 1 ? combine_kernel<1, 4>
                          : a.K == 2 ? combine_kernel<2, 2>
                                     : combine_kernel<4, 2>,
                          dim3(static_cast<unsigned>((pieces + per_cta - 1) / per_cta)),
                          dim3(kForwardThreads), 0, stream, a.rows, a.position, a.weights, a.out,
                          a.T, a.K, nch);
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, const DeviceInfo& dev,
                                    cudaStream_t stream) {
  const int nch = a.L / 8;
  // Two pieces per thread with few choices, where there are tokens enough for half the
  // threads (T = 512, K = 2, L = 2048: 2.9 us, 3.3 with half the threads).
  const int ahead = a.K <= 2 ? 2 : a.K <= 4 ? 4 : 8;
  const int spread = a.T < dev.num_sms * 4 ? 1 : pieces_ahead(ahead);
  const int per_thread = (nch + spread - 1) / spread;
  int tpt = 8;
  while (tpt < per_thread && tpt < kThreads) tpt *= 2;
  const int per_cta = kThreads / tpt;
  auto* k = ahead == 2   ? backward_kernel<2>(tpt)
            : ahead == 4 ? backward_kernel<4>(tpt)
                         : backward_kernel<8>(tpt);
  return launch_dependent(k, dim3((a.T + per_cta - 1) / per_cta), dim3(kThreads), 0, stream,
                          a.grad_out, a.rows, a.position, a.weights, a.grad_rows, a.grad_weights,
                          a.T, a.K, nch);
}

}  // namespace lt
