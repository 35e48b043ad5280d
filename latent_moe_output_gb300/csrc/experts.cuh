// Device helpers shared by the kernels of the bf16 experts: the table of the experts'
// rows, the activation with its derivative, and the 8-bit form of kept activations.
#pragma once

#include "block_launch.h"
#include "rows.cuh"

namespace lt {

// First row of each expert, from the caller's offsets: cut to [0, N] and to their running
// maximum, so that ones that run backwards give empty experts. Offsets that are null mean
// one matrix for all rows. Called by all threads; ends with a block barrier.
__device__ __forceinline__ void load_experts(const int32_t* offsets, int N, int E, int* s_first) {
  if (offsets != nullptr) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) s_first[e] = min(max(offsets[e], 0), N);
  } else if (threadIdx.x == 0) {
    s_first[0] = 0;
    s_first[1] = N;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int per = (E + 32) / 32;  // each lane takes a contiguous part
    const int lo = min(E + 1, lane * per), hi = min(E + 1, lo + per);
    int top = 0;
    for (int e = lo; e < hi; ++e) top = max(top, s_first[e]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, top, o);
      if (lane >= o) top = max(top, up);
    }
    int run = __shfl_up_sync(0xffffffffu, top, 1);
    if (lane == 0) run = 0;
    for (int e = lo; e < hi; ++e) s_first[e] = run = max(run, s_first[e]);
  }
  __syncthreads();
}

// s_unit[i], i = 0 .. count: the sum of units(j) over j < i. Called by all threads; ends
// with a block barrier.
template <typename Units>
__device__ __forceinline__ void sum_units(int count, int* s_unit, Units units) {
  for (int i = threadIdx.x; i < count; i += blockDim.x) s_unit[i] = units(i);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int per = (count + 32) / 32;  // each lane takes a contiguous part
    const int lo = min(count + 1, lane * per), hi = min(count + 1, lo + per);
    int sum = 0;
    for (int i = lo; i < min(hi, count); ++i) sum += s_unit[i];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    int run = incl - sum;
    for (int i = lo; i < hi; ++i) {
      const int own = i < count ? s_unit[i] : 0;
      s_unit[i] = run;
      run += own;
    }
  }
  __syncthreads();
}

// Experts by class, 8 first, then 7 .. 1, and by number within a class; those of class 0
// are left out. Returns how many there are. A warp places the experts of one class, so
// blocks of at least eight warps; called by all threads, ends with a block barrier.
constexpr int kClasses = 8;

template <typename Class>
__device__ __forceinline__ int order_experts(int E, int* s_order, Class class_of) {
  __shared__ int s_count[kClasses];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int count = 0;
  if (warp < kClasses) {
    for (int e = lane; e - lane < E; e += 32)
      count += __popc(__ballot_sync(0xffffffffu, e < E && class_of(e) == kClasses - warp));
    if (lane == 0) s_count[warp] = count;
  }
  __syncthreads();
  int at = 0, all = 0;
  for (int i = 0; i < kClasses; ++i) {
    if (i < warp) at += s_count[i];
    all += s_count[i];
  }
  if (warp < kClasses && count != 0) {
    for (int e = lane; e - lane < E; e += 32) {
      const bool mine = e < E && class_of(e) == kClasses - warp;
      const uint32_t who = __ballot_sync(0xffffffffu, mine);
      if (mine) s_order[at + __popc(who & ((1u << lane) - 1u))] = e;
      at += __popc(who);
    }
  }
  __syncthreads();
  return all;
}

// Bytes of shared memory for s_first, s_unit and s_order.
constexpr int experts_table_bytes(int E) { return ((E + 1) * 12 + 15) & ~15; }

// ------------------------------------------------------------ activation
// Both activations are g * sigmoid(s(g)): SiLU with s = g, the tanh form of GELU with
// s = sqrt(8 / pi) (g + 0.044715 g^3), as 0.5 (1 + tanh(y)) = sigmoid(2 y). The cubic
// takes g cut to +-32, where the sigmoid is 0 or 1 in FP32, so that it cannot overflow.
// (The division gives 0 for denominators past 2^126, where the sigmoid is below 2^-126.)
__device__ __forceinline__ float sigmoid(float s) {
  return __fdividef(1.f, 1.f + __expf(-s));
}

__device__ __forceinline__ float gelu_argument(float g) {
  const float c = fminf(fmaxf(g, -32.f), 32.f);
  return 1.59576912160573f * c * fmaf(0.044715f * c, c, 1.f);
}

template <int kAct>
__device__ __forceinline__ float activation(float g) {
  return g * sigmoid(kAct == kActSilu ? g : gelu_argument(g));
}

// The activation a and its derivative d at g.
template <int kAct>
__device__ __forceinline__ void activation_grad(float g, float& a, float& d) {
  const float s = sigmoid(kAct == kActSilu ? g : gelu_argument(g));
  a = g * s;
  float slope = 1.f;
  if (kAct != kActSilu) {
    const float c = fminf(fmaxf(g, -32.f), 32.f);
    slope = 1.59576912160573f * fmaf(3.f * 0.044715f * c, c, 1.f);
  }
  // s (1 - s) from the smaller of the two would keep more of the far tail, where the
  // product with g is below the rounding of the sum in 32 bits all the same.
  d = fmaf(a * (1.f - s), slope, s);
}

// ------------------------------------------------------------- 8-bit form
// 16 consecutive values share a power of two 2^(e - 127): the least e >= 1 for which the
// largest magnitude rounds to at most 127. An integer of 8 bits times a power of two is
// exact in bf16, so reading back adds no second rounding. e = 0 stands for a group of
// zeros, e = 255 for a group that holds an infinity or a NaN (read back as NaNs).
constexpr int kGroup8 = 16;

// `top`: the upper 16 bits of the largest magnitude (as bf16 has them; NaN sorts above
// infinity, and that above all). From 2^E up to 2^(E+1) it is 64 to 128 in units of
// 2^(E-6); from 127.5 on, where it rounds to 128, the next unit is taken. That is where the
// seven upper bits of the mantissa are ones, so adding one carries into the exponent.
__device__ __forceinline__ uint32_t exponent8(uint32_t top) {
  const int e = max(static_cast<int>((top + 1u) >> 7) - 6, 1);
  return top >= 0x7F80u ? 255u : top == 0u ? 0u : static_cast<uint32_t>(e);
}

// Factor from values to their integers; 0 for a group that is not finite.
__device__ __forceinline__ float scale8(uint32_t e) {
  return e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
}

// Adding 1.5 * 2^23 rounds to an integer (to nearest even) and leaves it, in two's
// complement, in the low bits.
constexpr float kToInteger = 12582912.f;

__device__ __forceinline__ uint8_t integer8(float v, uint32_t e) {
  const uint32_t w = __float_as_uint(fmaf(v, scale8(e), kToInteger));
  return static_cast<uint8_t>(e == 255u ? 0u : w & 0xFFu);
}

// Factor from integers back to values; NaN where e = 255 (0 times it is NaN).
__device__ __forceinline__ float unit8(uint32_t e) {
  return e == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e << 23);
}

}  // namespace lt
