// Activations in 8 bits, and the step of a gated block's gradient that reads them:
//   quantize8     per 16 columns e = the least exponent for which the largest magnitude
//                 rounds to at most 127 units of 2^(e-127), values = round(x / 2^(e-127))
//   dequantize8   values * 2^(e-127), exact in bf16
//   gated_grad    from kept projections g, u and dh: dg = dh u a'(g), du = dh a(g), and
//                 h = a(g) u again
// All three are bound by memory: every element is read and written once, a thread takes
// whole groups (16 columns; gated_grad 8 features of both projections), so that no value
// crosses lanes and an exponent is one byte load or store of neighbouring lanes.
// Measured: 16384 x 7168 in 54 us and back in 55 (6.7 TB/s, 99 % of a copy's rate); gated_grad
// of 65536 x 1024 from 8 bits in 106 (95 %). Sixteen features a thread, streaming stores and
// other block sizes were not faster.
// Rounding: h, dg and du go to bf16 once, as operands of the tensor cores.
#include "experts.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kThreads = 128;

// The integers of four values in one word.
__device__ __forceinline__ uint32_t integers4(float a, float b, float c, float d, float scale) {
  const uint32_t w0 = __float_as_uint(fmaf(a, scale, kToInteger));
  const uint32_t w1 = __float_as_uint(fmaf(b, scale, kToInteger));
  const uint32_t w2 = __float_as_uint(fmaf(c, scale, kToInteger));
  const uint32_t w3 = __float_as_uint(fmaf(d, scale, kToInteger));
  return __byte_perm(__byte_perm(w0, w1, 0x0040), __byte_perm(w2, w3, 0x0040), 0x5410);
}

// The four integers of a word as floats: a byte with its sign bit turned over is the
// integer plus 128, and behind 0x4B000000 it is 2^23 plus that.
__device__ __forceinline__ void floats4(uint32_t w, float (&v)[4]) {
  const uint32_t b = w ^ 0x80808080u;
  v[0] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7440)) - 8388736.f;
  v[1] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7441)) - 8388736.f;
  v[2] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7442)) - 8388736.f;
  v[3] = __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7443)) - 8388736.f;
}

// Largest magnitudes of the even and of the odd values of eight, in one word.
__device__ __forceinline__ uint32_t top_of(const uint4& v, uint32_t top) {
  top = __vmaxs2(top, v.x & 0x7FFF7FFFu);
  top = __vmaxs2(top, v.y & 0x7FFF7FFFu);
  top = __vmaxs2(top, v.z & 0x7FFF7FFFu);
  return __vmaxs2(top, v.w & 0x7FFF7FFFu);
}

// Group `i` of all rows: its first element and whether it has 16 columns (else 8).
struct Group {
  int64_t at;
  bool whole;
};

__device__ __forceinline__ Group group_at(int64_t i, int C) {
  if ((C & 15) == 0) return Group{i * 16, true};
  const int groups = (C + 15) / 16;
  const int64_t row = i >> 32 == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(groups)
                                   : i / groups;
  const int g = static_cast<int>(i - row * groups);
  return Group{row * C + g * 16, g + 1 < groups};
}

__global__ void __launch_bounds__(kThreads) quantize8_kernel(const Quantize8Args a) {
  pdl_wait();
  const int64_t groups = static_cast<int64_t>(a.T) * ((a.C + 15) / 16);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= groups) return;
  const Group g = group_at(i, a.C);
  const uint4* src = reinterpret_cast<const uint4*>(a.x + g.at);
  const uint4 lo = ld_stream_v4(src);
  const uint4 hi = g.whole ? ld_stream_v4(src + 1) : make_uint4(0, 0, 0, 0);
  float v[8], w[8];
  unpack8(lo, v);
  unpack8(hi, w);
  const uint32_t top = top_of(hi, top_of(lo, 0u));
  const uint32_t e = exponent8(max(top & 0xFFFFu, top >> 16));
  const float scale = scale8(e);
  uint4 q = make_uint4(integers4(v[0], v[1], v[2], v[3], scale),
                       integers4(v[4], v[5], v[6], v[7], scale),
                       integers4(w[0], w[1], w[2], w[3], scale),
                       integers4(w[4], w[5], w[6], w[7], scale));
  if (e == 255u) q = make_uint4(0, 0, 0, 0);
  int8_t* dst = a.values + g.at;
  if ((a.C & 15) == 0) {
    *reinterpret_cast<uint4*>(dst) = q;
  } else {  // rows begin at multiples of 8 bytes
    *reinterpret_cast<uint2*>(dst) = make_uint2(q.x, q.y);
    if (g.whole) *reinterpret_cast<uint2*>(dst + 8) = make_uint2(q.z, q.w);
  }
  a.exponents[i] = static_cast<uint8_t>(e);
}

__global__ void __launch_bounds__(kThreads) dequantize8_kernel(const Quantize8Args a) {
  pdl_wait();
  const int64_t groups = static_cast<int64_t>(a.T) * ((a.C + 15) / 16);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= groups) return;
  const Group g = group_at(i, a.C);
  const int8_t* src = a.values + g.at;
  uint4 q;
  if ((a.C & 15) == 0) {
    q = *reinterpret_cast<const uint4*>(src);
  } else {
    const uint2 lo = *reinterpret_cast<const uint2*>(src);
    const uint2 hi = g.whole ? *reinterpret_cast<const uint2*>(src + 8) : make_uint2(0, 0);
    q = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  const float unit = unit8(a.exponents[i]);
  const uint32_t words[4] = {q.x, q.y, q.z, q.w};
  uint32_t out[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[4];
    floats4(words[j], v);
    out[2 * j] = pack_bf16x2(v[0] * unit, v[1] * unit);
    out[2 * j + 1] = pack_bf16x2(v[2] * unit, v[3] * unit);
  }
  uint4* dst = reinterpret_cast<uint4*>(a.out + g.at);
  st_stream_v4(dst, make_uint4(out[0], out[1], out[2], out[3]));
  if (g.whole) st_stream_v4(dst + 1, make_uint4(out[4], out[5], out[6], out[7]));
}

// Eight kept values of one projection.
template <bool k8>
__device__ __forceinline__ void kept8(const GatedGradArgs& a, int64_t row2, int f, float (&v)[8]) {
  if constexpr (k8) {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.saved) +
                                                    row2 * a.F + f);
    const float unit = unit8(a.exponents[row2 * ((a.F + 15) / 16) + f / kGroup8]);
    float lo[4], hi[4];
    floats4(q.x, lo);
    floats4(q.y, hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = lo[j] * unit;
      v[4 + j] = hi[j] * unit;
    }
  } else {
    unpack8(ld_stream_v4(static_cast<const uint16_t*>(a.saved) + row2 * a.F + f), v);
  }
}

template <bool k8, int kAct>
__global__ void __launch_bounds__(kThreads) gated_grad_kernel(const GatedGradArgs a) {
  __shared__ int s_end;
  pdl_wait();
  int first = 0, end = a.N;
  if (a.offsets != nullptr) {
    // The first row that an expert owns and the one behind the last: offsets are cut to
    // [0, N] and to their running maximum.
    if (threadIdx.x == 0) s_end = 0;
    __syncthreads();
    int top = 0;
    for (int e = threadIdx.x; e <= a.E; e += kThreads)
      top = max(top, min(max(a.offsets[e], 0), a.N));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) atomicMax(&s_end, top);
    __syncthreads();
    first = min(max(a.offsets[0], 0), a.N);
    end = s_end;
  }
  const int vecs = a.F / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = i >> 32 == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(vecs)
                                   : i / vecs;
  if (row >= a.N) return;
  const int f = static_cast<int>(i - row * vecs) * 8;
  if (row < first || row >= end) {  // (the products read no gradient of these rows)
    if (a.hidden != nullptr)
      *reinterpret_cast<uint4*>(a.hidden + row * a.F + f) = make_uint4(0, 0, 0, 0);
    return;
  }
  float g[8], u[8], d[8];
  kept8<k8>(a, 2 * row, f, g);
  kept8<k8>(a, 2 * row + 1, f, u);
  if (a.grad_pre != nullptr) unpack8(ld_stream_v4(a.grad_hidden + row * a.F + f), d);
  float act[8], slope[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) activation_grad<kAct>(g[j], act[j], slope[j]);
  if (a.grad_pre != nullptr) {
    float dg[8], du[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dg[j] = d[j] * slope[j] * u[j];  // (a' is 0 far out, where d u may pass FP32's range)
      du[j] = d[j] * act[j];
    }
    uint16_t* dst = a.grad_pre + row * 2 * a.F + f;
    *reinterpret_cast<uint4*>(dst) = pack8(dg);
    *reinterpret_cast<uint4*>(dst + a.F) = pack8(du);
  }
  if (a.hidden != nullptr) {
    float h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = act[j] * u[j];
    *reinterpret_cast<uint4*>(a.hidden + row * a.F + f) = pack8(h);
  }
}

dim3 grid_of(int64_t items) {
  return dim3(static_cast<unsigned>((items + kThreads - 1) / kThreads));
}

}  // namespace

cudaError_t launch_quantize8(const Quantize8Args& a, const DeviceInfo&, cudaStream_t stream) {
  return launch_dependent(quantize8_kernel, grid_of(static_cast<int64_t>(a.T) * ((a.C + 15) / 16)),
                          dim3(kThreads), 0, stream, a);
}

cudaError_t launch_dequantize8(const Quantize8Args& a, const DeviceInfo&, cudaStream_t stream) {
  return launch_dependent(dequantize8_kernel,
                          grid_of(static_cast<int64_t>(a.T) * ((a.C + 15) / 16)), dim3(kThreads), 0,
                          stream, a);
}

cudaError_t launch_gated_grad(const GatedGradArgs& a, const DeviceInfo&, cudaStream_t stream) {
  const dim3 grid = grid_of(static_cast<int64_t>(a.N) * (a.F / 8));
  const bool k8 = a.saved_kind == kSaved8, silu = a.act == kActSilu;
  return launch_dependent(k8 ? silu ? gated_grad_kernel<true, kActSilu>
                                    : gated_grad_kernel<true, kActGelu>
                             : silu ? gated_grad_kernel<false, kActSilu>
                                    : gated_grad_kernel<false, kActGelu>,
                          grid, dim3(kThreads), 0, stream, a);
}

}  // namespace lt
