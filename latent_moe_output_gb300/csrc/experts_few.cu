// The products of experts.cu for calls of few rows, where reading the weights bounds the
// call and tiles of 256 weight rows would leave most SMs idle:
//   gated  h[r,f] = a(sum_c x[r,c] W_e[f,c]) * sum_c x[r,c] W_e[F+f,c]
//   rows   y[r,m] = sum_c x[r,c] W_e[m,c]
// A CTA takes 32 weight rows (gated: the gate and up rows of 16 features) against up to 8
// kTiles rows of one expert; its 16 warps split the columns and add up through shared
// memory in the order of the warps. Products are mma.sync m16n8k16: few rows cannot feed a
// tcgen05 tile, and the call waits for memory. The weights go from global memory straight
// into fragments: a lane reads 16 bytes, eight columns, of weight rows g and g + 8 and of
// row g of x. Which of the 16 columns of a fragment a value stands for does not matter as
// long as both operands agree, so the eight columns of a lane are its columns of two
// fragments, and no shuffle or shared memory lies between a load and its product. In the
// gated form fragment row g is a gate row and g + 8 the up row of the same feature.
// Two fragments of rows take all 128 registers that 512 threads leave, and spill one or two.
// Measured: one row of 7168 against 2 x 2048 weight rows 11.6 us, 75 % of a copy's rate (one
// wave of 128 CTAs, 2 to 3 us of it to begin and end); half as many loads in flight per lane
// 16.0, an L2 prefetch of the weights before the wait for the kernel before 13.7 against 12.5
// where they come from memory.
#include "experts.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kM = 2;                 // fragments of 16 weight rows per warp
constexpr int kRowsPerCta = 16 * kM;  // weight rows
constexpr int kUnroll = 2;            // 32 columns each, loaded ahead of their products
constexpr int kSpan = 32 * kUnroll;   // columns of a warp's turn

struct Params {
  const uint16_t* x;
  const uint16_t* weights;
  const int32_t* offsets;
  uint16_t* out;       // gated: [N,F], else [N,M]
  void* saved;         // gated: [N,2,F] or null
  uint8_t* exponents;
  int N, E;
  int M;               // columns of out
  int C;
  int saved_kind;
  int act;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool kGated, int kTiles>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const Params p) {
  constexpr int kTokens = 8 * kTiles;
  constexpr int kPitch = kTokens + 1;
  extern __shared__ int s_table[];
  __shared__ float sums[kWarps][kRowsPerCta * kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  int e = 0, row0 = 0, rows = p.N, before = 0, end = p.N, unit = blockIdx.y, units = 1;
  if (p.offsets != nullptr) {
    int* s_first = s_table;
    int* s_unit = s_first + p.E + 1;
    load_experts(p.offsets, p.N, p.E, s_first);
    sum_units(p.E, s_unit,
              [&](int i) { return (s_first[i + 1] - s_first[i] + kTokens - 1) / kTokens; });
    before = s_first[0];
    end = s_first[p.E];
    units = s_unit[p.E];
    if (unit < units) {
      int lo = 0, hi = p.E - 1;  // the expert with s_unit[e] <= unit < s_unit[e + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_unit[mid + 1] > unit)
          hi = mid;
        else
          lo = mid + 1;
      }
      e = lo;
      row0 = s_first[e] + (unit - s_unit[e]) * kTokens;
      rows = min(kTokens, s_first[e + 1] - row0);
    }
  } else {
    units = (p.N + kTokens - 1) / kTokens;
    row0 = unit * kTokens;
    rows = min(kTokens, p.N - row0);
  }
  const int f0 = blockIdx.x * (kGated ? kRowsPerCta / 2 : kRowsPerCta);

  if (unit < units) {
    const int g = lane >> 2, c4 = lane & 3;
    // Weight rows of the lane: fragment m, halves 0 and 1. Rows past the matrix repeat its
    // last one and are not stored.
    const uint16_t* w[kM][2];
    const size_t matrix = static_cast<size_t>(e) * (kGated ? 2 : 1) * p.M;
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = kGated ? f0 + m * 8 + g : f0 + m * 16 + h * 8 + g;
        const size_t r = matrix + min(f, p.M - 1) + (kGated && h ? p.M : 0);
        w[m][h] = p.weights + r * p.C + c4 * 8;
      }
    const uint16_t* x[kTiles];
    bool has[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      has[n] = n * 8 + g < rows;
      x[n] = p.x + static_cast<size_t>(row0 + (has[n] ? n * 8 + g : 0)) * p.C + c4 * 8;
    }
    float acc[kM][kTiles][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int c0 = warp * kSpan; c0 < p.C; c0 += kWarps * kSpan) {
      uint4 a[kUnroll][kM][2], b[kUnroll][kTiles];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + u * 32;
        const bool in = c + c4 * 8 < p.C;
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) a[u][m][h] = in ? ld_stream_v4(w[m][h] + c) : zero;
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
          b[u][n] = in && has[n] ? ld_global_v4(x[n] + c) : zero;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            mma_bf16(acc[m][n], a[u][m][0].x, a[u][m][1].x, a[u][m][0].y, a[u][m][1].y, b[u][n].x,
                     b[u][n].y);
            mma_bf16(acc[m][n], a[u][m][0].z, a[u][m][1].z, a[u][m][0].w, a[u][m][1].w, b[u][n].z,
                     b[u][n].w);
          }
    }
    // Element (j, lane) of a fragment: weight row g + 8 (j >> 1), row 2 c4 + (j & 1) of x.
    // In shared memory: row f of the features' gates, then of their ups.
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = kGated ? (j >> 1) * (kRowsPerCta / 2) + m * 8 + g
                               : m * 16 + (j >> 1) * 8 + g;
          sums[warp][r * kPitch + n * 8 + c4 * 2 + (j & 1)] = acc[m][n][j];
        }
    __syncthreads();
    auto total = [&](int r, int t) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) v += sums[q][r * kPitch + t];
      return v;
    };
    if constexpr (kGated) {
      constexpr int kF = kRowsPerCta / 2;
      for (int i = threadIdx.x; i < kF * kTokens; i += kThreads) {
        const int f = i % kF, t = i / kF;  // (half a warp has the 16 features of one row)
        const float gate = total(f, t), up = total(kF + f, t);
        const bool live = t < rows && f0 + f < p.M;
        const size_t row = static_cast<size_t>(row0) + t;
        const float h = (p.act == kActSilu ? activation<kActSilu>(gate)
                                           : activation<kActGelu>(gate)) * up;
        if (live) p.out[row * p.M + f0 + f] = static_cast<uint16_t>(pack_bf16x2(h, 0.f));
        if (p.saved_kind == kSavedBf16) {
          if (live) {
            uint16_t* k = static_cast<uint16_t*>(p.saved) + row * 2 * p.M + f0 + f;
            k[0] = static_cast<uint16_t>(pack_bf16x2(gate, 0.f));
            k[p.M] = static_cast<uint16_t>(pack_bf16x2(up, 0.f));
          }
        } else if (p.saved_kind == kSaved8) {
          // Both maxima in one word; a group is half a warp.
          uint32_t top = f0 + f < p.M ? __byte_perm(__float_as_uint(gate), __float_as_uint(up),
                                                    0x7632) & 0x7FFF7FFFu
                                      : 0u;
#pragma unroll
          for (int o = 1; o < 16; o <<= 1)
            top = __vmaxs2(top, __shfl_xor_sync(0xffffffffu, top, o));
          const uint32_t e0 = exponent8(top & 0xFFFFu), e1 = exponent8(top >> 16);
          if (live) {
            uint8_t* k = static_cast<uint8_t*>(p.saved) + row * 2 * p.M + f0 + f;
            k[0] = integer8(gate, e0);
            k[p.M] = integer8(up, e1);
            if (f == 0) {
              const int groups = (p.M + kGroup8 - 1) / kGroup8;
              uint8_t* at = p.exponents + row * 2 * groups + f0 / kGroup8;
              at[0] = static_cast<uint8_t>(e0);
              at[groups] = static_cast<uint8_t>(e1);
            }
          }
        }
      }
    } else {
      for (int i = threadIdx.x; i < kRowsPerCta * kTokens; i += kThreads) {
        const int m = i % kRowsPerCta, t = i / kRowsPerCta;
        const float v = total(m, t);
        if (t < rows && f0 + m < p.M)
          p.out[(static_cast<size_t>(row0) + t) * p.M + f0 + m] =
              static_cast<uint16_t>(pack_bf16x2(v, 0.f));
      }
    }
  }
  pdl_launch_dependents();
  // Rows that no expert owns, over the CTAs that are last in the order of units.
  const int none = before + p.N - end;
  if (none == 0) return;
  const int ctas = static_cast<int>(gridDim.x * gridDim.y);
  const int me = ctas - 1 - static_cast<int>(blockIdx.y * gridDim.x + blockIdx.x);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int i = me; i < none; i += ctas) {
    const size_t r = static_cast<size_t>(i < before ? i : end + (i - before));
    uint4* o = reinterpret_cast<uint4*>(p.out + r * p.M);
    for (int c = threadIdx.x; c < p.M / 8; c += kThreads) o[c] = zero;
    if (kGated && p.saved_kind != kSavedNone) {
      const int bytes = (p.saved_kind == kSavedBf16 ? 4 : 2) * p.M;
      uint4* k = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.saved) + r * bytes);
      for (int c = threadIdx.x; c < bytes / 16; c += kThreads) k[c] = zero;
      if (p.saved_kind == kSaved8) {
        const int groups = 2 * ((p.M + kGroup8 - 1) / kGroup8);
        for (int c = threadIdx.x; c < groups; c += kThreads) p.exponents[r * groups + c] = 0;
      }
    }
  }
}

typedef void (*Kernel)(const Params);

template <bool kGated>
cudaError_t launch(const Params& p, cudaStream_t stream) {
  // Rows that an expert has on average bound the tiles of a pass.
  const int mean = p.offsets == nullptr ? p.N : (p.N + p.E - 1) / p.E;
  const int tiles = mean > 8 ? 2 : 1;
  const Kernel kernel = tiles == 2 ? few_kernel<kGated, 2> : few_kernel<kGated, 1>;
  const int per = kGated ? kRowsPerCta / 2 : kRowsPerCta;
  const int units = p.offsets == nullptr ? (p.N + 8 * tiles - 1) / (8 * tiles)
                                         : std::min(p.N, p.E + p.N / (8 * tiles));
  return launch_dependent(kernel, dim3((p.M + per - 1) / per, units), dim3(kThreads),
                          p.offsets == nullptr ? 0 : experts_table_bytes(p.E), stream, p);
}

}  // namespace

// Two waves of CTAs for rows of several experts (8 of 256 experts of 2 x 1024 x 2048, 512
// CTAs: 24 us against 20 of the tensor-core kernel; 2 tokens with 4 of 32 experts of 2 x 512
// x 2048, 256 CTAs: 11.6 against 13.1; 8 with 4 of 8, 2 x 256 x 1024: 6.7 against 9.2). With
// one matrix, 16 rows a pass, of which
// all but the first read the weights from L2: the passes' time at 6.8 TB/s against that of
// the tensor-core kernel, 1.5 us more to begin with and 0.2 us per 128 columns (both
// measured, us: 58.7 MB of weights, 16 and 24 rows 13.5 and 20 against 16.7; 29 MB, 16 rows
// 6.9 against 10.3; 4.2 MB, 64 rows 6.6 against 8.8).
bool few_rows(const int32_t* offsets, int N, int E, int M, int C, bool gated,
              const DeviceInfo& dev) {
  const int64_t per = gated ? kRowsPerCta / 2 : kRowsPerCta;
  const int64_t blocks = (M + per - 1) / per;
  if (offsets != nullptr) return N <= 32 && std::min(N, E) * blocks <= 2 * dev.num_sms;
  const double passes = (N + 15) / 16;
  const double bytes = (gated ? 4.0 : 2.0) * M * C;
  return N <= 64 && passes * bytes / 6.8e6 <= 1.5 + 0.2 * ((C + 127) / 128);
}

cudaError_t launch_expert_gated_few(const ExpertGatedArgs& a, cudaStream_t stream) {
  const Params p{a.x, a.weights, a.offsets, a.hidden, a.saved, a.exponents, a.N, a.E, a.F, a.C,
                 a.saved_kind, a.act};
  return launch<true>(p, stream);
}

cudaError_t launch_expert_rows_few(const ExpertRowsArgs& a, cudaStream_t stream) {
  const Params p{a.x, a.weights, a.offsets, a.out, nullptr, nullptr, a.N, a.E, a.M, a.K,
                 kSavedNone, kActSilu};
  return launch<false>(p, stream);
}

}  // namespace lt
