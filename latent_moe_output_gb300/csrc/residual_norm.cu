// latent_tail_residual_norm and its gradient: the norm after a block, its gate,
// the scaled residual sum and the norm before the next block.
//
//   u = y * r1 * gp,  r1 = rsqrt(mean y^2 + eps)        (y itself without gp)
//   v = s * x + gate * u
//   z = v * r2 * gn,  r2 = rsqrt(mean v^2 + eps)
//
// Gradient, from dv (of v as an output) and dz:
//   a  = dz * gn,   d  = dv + r2 * (a - vh * mean(a * vh)),  vh = v * r2
//   dx = s * d,     dgate = d * u,   b = d * gate * gp
//   dy = r1 * (b - yh * mean(b * yh)),  yh = y * r1
//   dgp = sum_t d * gate * yh,  dgn = sum_t dz * vh
//
// Every element is read once and written once, so memory bounds both. Measured at
// T = 8192, H = 7168, bf16 (GB300, calls back to back): forward 72 us = 6.6 TB/s, 97 % of
// the measured copy rate; gradient 110 us = 6.4 TB/s, 94 %. One row alone: 3.6 us.
#include "block_launch.h"
#include "rows.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kMaxThreads = 512;
// Column sum: threads per CTA, and the widest rows for 4 float4 columns per CTA instead
// of 16 (T = 8192 / T = 1000, gradient in us with 4 and with 16: H = 1024 23.0 / 8.8 and
// 26.0 / 11.8, H = 4000 72.6 / 17.0 and 73.1 / 18.2; H = 7168 at T = 4000 59.6 and 58.2).
constexpr int kReduceThreads = 512;
constexpr int kReduceNarrowH = 4096;

struct Shape {
  int threads;  // per CTA
  int tpr;      // threads per token row (whole warps)
  int per_cta;  // token rows a CTA works on at once
  int pieces;   // 8-element pieces per thread
};

Shape shape_of(int H) {
  const int nch = H / 8;
  Shape s;
  // A warp takes a row of up to 64 pieces (T = 8192, H = 264: 6.3 us, 7.8 with two warps;
  // H = 512: 7.9 and 9.2).
  s.pieces = nch <= 32 ? 1 : nch <= 64 ? 2 : nch <= 256 ? 1 : 2;
  if (nch <= 128) {
    s.tpr = nch <= 64 ? 32 : 128;
    s.threads = 256;
  } else {
    s.tpr = ((nch + s.pieces - 1) / s.pieces + 31) / 32 * 32;
    s.threads = s.tpr;
  }
  s.per_cta = s.threads / s.tpr;
  return s;
}

// Sum over the threads of a row. `red` holds one value per warp; consecutive
// calls alternate between two of them, so one barrier per call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int row_in_cta, int warps_per_row) {
  v = warp_sum_f(v);
  if (warps_per_row == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum_f(lane < warps_per_row ? red[row_in_cta * warps_per_row + lane] : 0.f);
}

__device__ __forceinline__ void load8(const float* p, float (&a)[8]) {
  const float4 lo = __ldg(reinterpret_cast<const float4*>(p));
  const float4 hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
  a[0] = lo.x; a[1] = lo.y; a[2] = lo.z; a[3] = lo.w;
  a[4] = hi.x; a[5] = hi.y; a[6] = hi.z; a[7] = hi.w;
}

// Eight elements of the residual stream, bf16 or FP32.
template <bool kF32>
__device__ __forceinline__ void load_res8(const void* base, size_t at, float (&a)[8]) {
  if constexpr (kF32) {
    const float* p = static_cast<const float*>(base) + at;
    const uint4 lo = ld_once_v4(p), hi = ld_once_v4(p + 4);
    a[0] = __uint_as_float(lo.x); a[1] = __uint_as_float(lo.y);
    a[2] = __uint_as_float(lo.z); a[3] = __uint_as_float(lo.w);
    a[4] = __uint_as_float(hi.x); a[5] = __uint_as_float(hi.y);
    a[6] = __uint_as_float(hi.z); a[7] = __uint_as_float(hi.w);
  } else {
    unpack8(ld_once_v4(static_cast<const uint16_t*>(base) + at), a);
  }
}

template <bool kF32>
__device__ __forceinline__ void store_res8(void* base, size_t at, const float (&a)[8]) {
  if constexpr (kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(a[0], a[1], a[2], a[3]);
    p[1] = make_float4(a[4], a[5], a[6], a[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(a);
  }
}

// The same on register pairs; 32 bytes of FP32 at a time.
__device__ __forceinline__ void pairs_of(const float4& lo, const float4& hi, f32x2 (&a)[4]) {
  a[0] = pair(lo.x, lo.y);
  a[1] = pair(lo.z, lo.w);
  a[2] = pair(hi.x, hi.y);
  a[3] = pair(hi.z, hi.w);
}
__device__ __forceinline__ void load8(const float* p, f32x2 (&a)[4]) {
  pairs_of(__ldg(reinterpret_cast<const float4*>(p)), __ldg(reinterpret_cast<const float4*>(p) + 1),
           a);
}
__device__ __forceinline__ void store8(float* p, const f32x2 (&a)[4]) {
  ulonglong2* q = reinterpret_cast<ulonglong2*>(p);
  q[0] = make_ulonglong2(a[0], a[1]);
  q[1] = make_ulonglong2(a[2], a[3]);
}
template <bool kF32>
__device__ __forceinline__ void store_res8(void* base, size_t at, const f32x2 (&a)[4]) {
  if constexpr (kF32)
    store8(static_cast<float*>(base) + at, a);
  else
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(a);
}

__device__ __forceinline__ void gate8(const void* gate, int kind, int t, int col, size_t at,
                                      float (&a)[8]) {
  if (kind == kGateFull) {
    unpack8(ld_stream_v4(static_cast<const uint16_t*>(gate) + at), a);
  } else if (kind == kGateChannel) {
    load8(static_cast<const float*>(gate) + col, a);
  } else {
    const float g = kind == kGateToken ? __ldg(static_cast<const float*>(gate) + t) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = g;
  }
}

template <bool kF32>
struct Raw;
template <>
struct Raw<false> {
  uint4 v;
  __device__ __forceinline__ void load(const void* base, size_t at) {
    v = ld_once_v4(static_cast<const uint16_t*>(base) + at);
  }
  __device__ __forceinline__ void get(float (&a)[8]) const { unpack8(v, a); }
};
template <>
struct Raw<true> {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void* base, size_t at) {
    lo = ld_once_v4(static_cast<const float*>(base) + at);
    hi = ld_once_v4(static_cast<const float*>(base) + at + 4);
  }
  __device__ __forceinline__ void get(float (&a)[8]) const {
    a[0] = __uint_as_float(lo.x); a[1] = __uint_as_float(lo.y);
    a[2] = __uint_as_float(lo.z); a[3] = __uint_as_float(lo.w);
    a[4] = __uint_as_float(hi.x); a[5] = __uint_as_float(hi.y);
    a[6] = __uint_as_float(hi.z); a[7] = __uint_as_float(hi.w);
  }
};

// One row per group of `tpr` threads. A row's loads, two reductions and stores
// follow one another, so several CTAs per SM keep the memory busy; rows are held
// as they were loaded to keep the registers for that.
template <int kPieces, bool kF32>
__global__ void __launch_bounds__(kMaxThreads, 2)
    residual_norm_kernel(const ResidualNormArgs a, int tpr) {
  __shared__ float red[2][kMaxThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int row = threadIdx.x / tpr, lane = threadIdx.x - row * tpr, wpr = tpr >> 5;
  const int t = blockIdx.x * (blockDim.x / tpr) + row;
  const bool live = t < a.T;
  const size_t base = static_cast<size_t>(t) * a.H;
  const float inv_h = 1.0f / static_cast<float>(a.H);

  uint4 y[kPieces];
  Raw<kF32> x[kPieces];
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
    if (live && col < a.H) {
      y[q] = ld_stream_v4(a.block + base + col);
      x[q].load(a.residual, base + col);
    } else {
      y[q] = make_uint4(0, 0, 0, 0);
    }
  }
  float r1 = 1.f, ss = 0.f;
  if (a.post != nullptr) {
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      float f[8];
      unpack8(y[q], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
    }
    r1 = 1.0f / sqrtf(row_sum(ss, red[0], row, wpr) * inv_h + a.eps);
  }
  ss = 0.f;
  float v[kPieces][8];
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[q][i] = 0.f;
    if (live && col < a.H) {
      float u[8], w[8];
      unpack8(y[q], u);
      if (a.post != nullptr) {
        load8(a.post + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = u[i] * r1 * w[i];
      }
      gate8(a.gate, a.gate_kind, t, col, base + col, w);
      x[q].get(v[q]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[q][i] = fmaf(w[i], u[i], a.scale * v[q][i]);
      store_res8<kF32>(a.residual_out, base + col, v[q]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[q][i], v[q][i], ss);
  }
  if (a.next == nullptr) return;
  const float r2 = 1.0f / sqrtf(row_sum(ss, red[1], row, wpr) * inv_h + a.eps);
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
    if (live && col < a.H) {
      float w[8];
      load8(a.next + col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[q][i] * r2 * w[i];
      *reinterpret_cast<uint4*>(a.next_out + base + col) = pack8(w);
    }
  }
}

// ------------------------------------------------------------ ring kernel
// The gradient for H > 512: one to six CTAs per SM walk over token rows, one or two
// 8-element pieces of the row per thread. The rows (up to five arrays) come through
// a ring of stages with bulk copies that run ahead of the arithmetic; a stage is
// refilled once all threads are past the next row's barrier. Above H = 8192 the sums over
// tokens no longer fit in one SM's registers: a cluster of two CTAs then shares each
// row, half of the columns each, and exchanges the row's partial sums through
// distributed shared memory.
constexpr int kNarrowMaxH = 512;  // up to here a warp takes a row of the gradient
constexpr int kRingMinH = kNarrowMaxH + 8, kRingMaxH = 8192;  // per CTA
constexpr int kRingMaxStages = 6;
// Forward: fewest token rows per SM up to kRingMaxH (T = 456, H = 7168: 6.7 us, 8.2 with
// the direct kernel; T = 200: 4.1 and 4.6; T = 100, H = 8192: 4.8 and 4.4). Wider rows
// always take the ring (T = 100, H = 9152: 3.5 us, 5.1 with a direct kernel; T = 1, H =
// 16384: 4.8 and 5.9), with a single stage if two do not fit (T = 1700, H = 16384, FP32,
// full gate: 82 and 86).
constexpr int kRingMinRowsPerSm = 1;
constexpr size_t kRingSmem = 224 * 1024;  // one CTA per SM
// Narrower rows take a warp each (T = 8192, us direct and ring: H = 512 7.9 and 9.9, 520
// 10.9 and 9.5, 1024 16.9 and 13.5, 2048 31.8 and 22.8, 3584 49.5 and 38.5).
constexpr int kForwardRingMinH = 520;
constexpr int kForwardRingBytes = 112 * 1024;  // per SM
// Rings of few threads let the next kernel's CTAs in when they are done (T = 8192, H = 520
// and 1024: 10.5 and 13.5 us, 12.4 and 14.4 when at once; wider rows the other way round,
// H = 2560: 29.9 and 29.5).
constexpr int kLateTriggerThreads = 288;

// Rows of few pieces have few threads: several CTAs then share an SM.
constexpr int ring_ctas_per_sm(int threads) {
  return threads <= 128 ? 6 : threads <= 288 ? 3 : threads <= 448 ? 2 : 1;
}
// CTAs that share a row, and the columns of the first of them.
constexpr int ring_cluster(int H) { return H > kRingMaxH ? 2 : 1; }
constexpr int ring_width(int H) { return ring_cluster(H) == 1 ? H : (H / 8 + 1) / 2 * 8; }

constexpr int ring_threads(int H) { return (H / 8 + 31) / 32 * 32; }
// The forward ring: one piece per thread up to 1024 threads, else two.
constexpr int forward_ring_threads(int H) {
  return H <= kRingMaxH ? ring_threads(H) : (H / 8 + 63) / 64 * 32;
}

// CTAs per SM, within 72 registers per thread (8192 rows of H = 768: 10.9 us with eight
// of 96 threads, 12.5 with six).
constexpr int forward_ring_ctas(int threads) {
  return threads <= 96 ? 8 : threads <= 128 ? 6 : threads <= 288 ? 3 : threads <= 448 ? 2 : 1;
}

// The gradient's ring: rows of more than 448 pieces take two per thread (half the
// warps to synchronize and to reduce over, with twice the work each).
constexpr int backward_ring_pieces(int H) { return H / 8 > 448 ? 2 : 1; }
constexpr int backward_ring_threads(int H) {
  const int per_thread = backward_ring_pieces(H);
  return ((H / 8 + per_thread - 1) / per_thread + 31) / 32 * 32;
}
constexpr int backward_ring_ctas(int H) {
  return backward_ring_pieces(H) == 2 ? 1 : ring_ctas_per_sm(ring_threads(H));
}
constexpr size_t backward_ring_smem(int H) {
  return backward_ring_ctas(H) == 1 ? kRingSmem : kRingSmem / backward_ring_ctas(H) - 2048;
}

// Dynamic shared memory with which `ctas` CTAs of a ring kernel are resident on an SM:
// 228 KB, of which a CTA also takes its static arrays and 1 KB of the system's.
constexpr size_t kSmemOfSm = 228 * 1024;
constexpr size_t kForwardStatic = 640, kBackwardStatic = 2176;
constexpr size_t resident_smem(int ctas, size_t static_bytes) {
  return kSmemOfSm / ctas - static_bytes - 1024;
}

// Stages of the forward ring: two, three while they stay within kForwardRingBytes (T =
// 8192, H = 7168, channel gate: 75 us with two and 82 with three; H = 4096 47 and 43; T =
// 4000, H = 10240 54 and 57; H = 9152 50 and 47).
constexpr int forward_ring_stages(int H, int stage_bytes) {
  const int ctas = forward_ring_ctas(forward_ring_threads(H));
  const size_t smem = ctas == 1 ? kRingSmem : kRingSmem / ctas - 2048;
  const int stages = std::min(3, std::max(2, kForwardRingBytes / ctas / stage_bytes));
  return static_cast<int>(std::min<size_t>(stages, smem / stage_bytes));
}

// Bytes of `rows` token rows in the forward ring: two bytes per element and `halves`
// (block 1, residual 1 or 2, a gate per element 1).
constexpr int forward_stage_bytes(int H, int halves, int rows) {
  return (rows * halves * 2 * H + 127) / 128 * 128;
}
// Token rows that the forward ring takes at a time: two, where two stages of them fit.
constexpr int forward_ring_rows(int H, int halves) {
  return H <= kRingMaxH && forward_ring_stages(H, forward_stage_bytes(H, halves, 2)) >= 2 ? 2 : 1;
}
// Up to kRingMaxH only FP32 rows with a gate per element are taken singly, and those in
// CTAs of two sizes: no kernel is built for others.
constexpr bool single_rows_as_built() {
  for (int H = kForwardRingMinH; H <= kRingMaxH; H += 8)
    for (int halves = 2; halves <= 4; ++halves) {
      const int threads = forward_ring_threads(H);
      if (forward_ring_rows(H, halves) == 1 &&
          (halves != 4 || !((threads > 288 && threads <= 448) || threads > 896)))
        return false;
    }
  return true;
}
static_assert(single_rows_as_built(), "forward_ring_kernel lacks a kernel");

// Stages of the gradient's ring: three where they fit; more only while they leave 24 KB of
// the SM's shared memory to the L1 cache (T = 8192, H = 7168: 110 us with three stages, 121
// with four, 154 with two; T = 777, H = 5128, FP32, full gate: 23.1 with three, 26.3 with
// two); fewer where not all CTAs of the SM would be resident (T = 8192, FP32: H = 1000 30.3
// us with two, 34.5 with three and a CTA that waits; H = 856, full gate, 30.9 and 35.4).
constexpr int backward_ring_stages(int width, int stage_bytes) {
  const size_t smem = backward_ring_smem(width);
  int stages = static_cast<int>(std::min<size_t>(kRingMaxStages, smem * 25 / 28 / stage_bytes));
  stages = std::max(stages, static_cast<int>(std::min<size_t>(3, smem / stage_bytes)));
  return std::min(stages, static_cast<int>(
                              resident_smem(backward_ring_ctas(width), kBackwardStatic) /
                              stage_bytes));
}

// Whether the CTAs that calls of any width launch per SM are all resident: for FP32 (r = 2)
// and bf16 rows of 1 to 3 (forward) and 2 to 5 arrays.
constexpr bool rings_resident() {
  for (int H = kRingMinH; H <= kRingMaxH; H += 8)
    for (int halves = 2; halves <= 7; ++halves) {  // bytes of a row's arrays / 2 H
      const int bytes = (halves * 2 * H + 127) / 128 * 128;
      const int forward = forward_ring_ctas(forward_ring_threads(H));
      const int backward = backward_ring_ctas(H);
      if (backward_ring_stages(H, bytes) * bytes >
          static_cast<int>(resident_smem(backward, kBackwardStatic)))
        return false;
      if (halves <= 4)
        for (int rows = 1; rows <= 2; ++rows) {
          const int stage = forward_stage_bytes(H, halves, rows);
          if (forward_ring_stages(H, stage) * stage >
              static_cast<int>(resident_smem(forward, kForwardStatic)))
            return false;
        }
    }
  return true;
}
static_assert(rings_resident(), "CTAs of a ring kernel that are launched together fit an SM");

// Sums of 1, 2, 4 or 8 values over the CTA, or the cluster of two, with one barrier:
// halving exchanges leave a lane with a part of one value, one partial per warp goes to
// shared memory (of both CTAs), and each warp adds the warps' partials again. `red` is
// [kValues][32], zero where there is no warp; the CTAs of a cluster (of up to 16 warps
// each) have half of it each. Consecutive calls use different ones. With a CTA's abort flag:
// returns whether no thread had given up on a wait at the barrier (read beside the
// partials; after them it costs up to 7 % of a forward call).
template <int kValues, int kCluster>
__device__ __forceinline__ bool cta_sum(float (&v)[kValues], float (*red)[32],
                                        volatile int* abort_v = nullptr) {
  bool came = true;
  constexpr int kLanes = 32 / kValues;  // lanes per value
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[kValues];
#pragma unroll
  for (int i = 0; i < kValues; ++i) w[i] = v[i];
#pragma unroll
  for (int n = kValues / 2, o = 16; n > 0; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i)
      w[i] = (up ? w[n + i] : w[i]) + __shfl_xor_sync(0xffffffffu, up ? w[i] : w[n + i], o);
  }
  float c = w[0];
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  const int which = lane / kLanes, at = (lane % kLanes) * kValues;
  if constexpr (kCluster == 1) {
    if (lane % kLanes == 0) red[which][warp] = c;
    __syncthreads();
    if (abort_v != nullptr) came = !*abort_v;
  } else {
    const uint32_t rank = cluster_rank();
    if (lane % kLanes == 0) {
      float* own = &red[which][rank * 16 + warp];
      *own = c;
      st_dsmem_f32(map_to_rank(smem_u32(own), rank ^ 1u), c);
    }
    cluster_sync();
  }
  c = 0.f;
  if constexpr (kValues >= 4) {
#pragma unroll
    for (int i = 0; i < kValues; i += 4) {
      const float4 p = *reinterpret_cast<const float4*>(&red[which][at + i]);
      c += (p.x + p.y) + (p.z + p.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kValues; ++i) c += red[which][at + i];
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
#pragma unroll
  for (int i = 0; i < kValues; ++i) v[i] = __shfl_sync(0xffffffffu, c, kLanes * i);
  return came;
}

// The part of a row that a CTA of a cluster owns.
struct RowPart {
  int first, width;  // columns
};
template <int kCluster>
__device__ __forceinline__ RowPart row_part(int H) {
  if constexpr (kCluster == 1) return RowPart{0, H};
  const int half = (H / 8 + 1) / 2 * 8;
  return cluster_rank() == 0 ? RowPart{0, half} : RowPart{half, H - half};
}

// A thread's piece of a row in shared memory.
__device__ __forceinline__ void lds8(const float* row, int lane, f32x2 (&a)[4]) {
  pairs_of(*reinterpret_cast<const float4*>(row + lane * 8),
           *reinterpret_cast<const float4*>(row + lane * 8 + 4), a);
}
__device__ __forceinline__ void lds8(const uint8_t* row, int lane, f32x2 (&a)[4]) {
  unpack8(*reinterpret_cast<const uint4*>(row + lane * 16), a);
}
template <bool kF32>
__device__ __forceinline__ void lds_res8(const uint8_t* row, int lane, f32x2 (&a)[4]) {
  if constexpr (kF32)
    lds8(reinterpret_cast<const float*>(row), lane, a);
  else
    lds8(row, lane, a);
}

// ------------------------------------------------- arithmetic of the gradient
// What a row of the gradient needs besides its elements.
struct GradRow {
  float r1, r2, k2, by, gt;
};

// Which inputs a call has. The kernels are built for calls with all of them (kAll:
// without, kAllGated: with a gate per element), where the choices fold away, and for
// the rest.
struct GradHas {
  bool post, next, dv, full_gate;
};
enum GradMode { kSome = 0, kAll = 1, kAllGated = 2 };

template <int kMode>
__device__ __forceinline__ GradHas grad_has(const ResidualNormBackwardArgs& a) {
  if constexpr (kMode == kSome)
    return GradHas{a.post != nullptr, a.next != nullptr, a.grad_residual_out != nullptr,
                   a.gate_kind == kGateFull};
  return GradHas{true, true, true, kMode == kAllGated};
}

int grad_mode(const ResidualNormBackwardArgs& a) {
  if (a.post == nullptr || a.next == nullptr || a.grad_residual_out == nullptr) return kSome;
  return a.gate_kind == kGateFull ? kAllGated : kAll;
}

// Sums over one 8-element piece. With w = gp * gate: y y, v v, a v (a = dz gn), then
// the terms of mean(b yh), which is linear in d: dv w y, a w y, v w y. So one
// reduction per row is enough. gp holds a channel gate already.
__device__ __forceinline__ void grad_sums(f32x2 (&q)[6], const GradHas& has, const f32x2 (&y)[4],
                                          const f32x2 (&v)[4], const f32x2 (&z)[4],
                                          const f32x2 (&dv)[4], const f32x2 (&g)[4],
                                          const f32x2 (&gp)[4], const f32x2 (&gn)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[0] = fma2(y[i], y[i], q[0]);
    f32x2 wy = mul2(y[i], gp[i]);
    if (has.full_gate) wy = mul2(wy, g[i]);
    if (has.next) {
      const f32x2 a = mul2(z[i], gn[i]);
      q[1] = fma2(v[i], v[i], q[1]);
      q[2] = fma2(a, v[i], q[2]);
      q[4] = fma2(a, wy, q[4]);
      q[5] = fma2(v[i], wy, q[5]);
    }
    if (has.dv) q[3] = fma2(dv[i], wy, q[3]);
  }
}

// From the row's sums: d = dv + r2 a + k2 v, and by = r1 sum(d w y), a token gate apart.
__device__ __forceinline__ GradRow grad_row(const float (&sum)[8], const GradHas& has,
                                            float inv_h, float eps, float gt) {
  GradRow r;
  r.r1 = has.post ? rsqrtf(fmaf(sum[0], inv_h, eps)) : 1.f;
  r.r2 = has.next ? rsqrtf(fmaf(sum[1], inv_h, eps)) : 0.f;
  r.k2 = -(sum[2] * inv_h * r.r2 * r.r2 * r.r2);
  r.by = r.r1 * fmaf(r.k2, sum[5], fmaf(r.r2, sum[4], sum[3]));
  r.gt = gt;
  return r;
}

// One piece: dv becomes d, z becomes dx; acc_n += dz vh.
__device__ __forceinline__ void grad_residual_piece(const GradRow& r, const GradHas& has,
                                                    float scale, const f32x2 (&v)[4],
                                                    f32x2 (&z)[4], f32x2 (&dv)[4],
                                                    const f32x2 (&gn)[4], f32x2 (&acc_n)[4]) {
  const f32x2 r2 = both(r.r2), k2 = both(r.k2), s = both(scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (has.next) {
      const f32x2 zr = mul2(z[i], r2);
      dv[i] = fma2(zr, gn[i], fma2(k2, v[i], dv[i]));
      acc_n[i] = fma2(zr, v[i], acc_n[i]);
    }
    z[i] = mul2(s, dv[i]);
  }
}

// One piece: d becomes dy, g the gradient of a full gate; acc_p += d gate yh (d yh
// with a channel gate). dy = gt (r1 b - y r1^2 mean(b yh)) with b = d gate gp.
__device__ __forceinline__ void grad_block_piece(const GradRow& r, const GradHas& has,
                                                 float inv_h, const f32x2 (&y)[4],
                                                 f32x2 (&d)[4], f32x2 (&g)[4],
                                                 const f32x2 (&gp)[4], f32x2 (&acc_p)[4]) {
  const f32x2 c = both(r.r1 * r.gt);
  const f32x2 k = both(has.post ? -(r.by * inv_h * r.r1 * r.r1 * r.gt) : 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 e = mul2(d[i], c);
    if (has.full_gate) {
      const f32x2 b = mul2(e, gp[i]);
      acc_p[i] = fma2(mul2(e, g[i]), y[i], acc_p[i]);
      d[i] = mul2(b, g[i]);
      g[i] = mul2(b, y[i]);  // d u
    } else {
      acc_p[i] = fma2(e, y[i], acc_p[i]);
      d[i] = mul2(e, gp[i]);
    }
    if (has.post) d[i] = fma2(k, y[i], d[i]);
  }
}

// Weights of a piece for the two functions above; zeros the sums.
__device__ __forceinline__ void grad_weights(const ResidualNormBackwardArgs& a, int col, bool on,
                                             f32x2 (&gp)[4], f32x2 (&gn)[4], f32x2 (&acc_p)[4],
                                             f32x2 (&acc_n)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    gp[i] = both(1.f);
    gn[i] = acc_p[i] = acc_n[i] = both(0.f);
  }
  if (!on) return;
  if (a.post != nullptr) load8(a.post + col, gp);
  if (a.next != nullptr) load8(a.next + col, gn);
  if (a.gate_kind == kGateChannel) {
    f32x2 g[4];
    load8(static_cast<const float*>(a.gate) + col, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) gp[i] = mul2(gp[i], g[i]);
  }
}

// ------------------------------------------------- gradient of narrow rows
// H <= 512: one warp per token row, no barriers; the rows of a CTA's warps add up
// through shared memory at the end.
constexpr int kNarrowThreads = 256;
// CTAs per SM: rows of two pieces per thread take up to 191 registers.
constexpr int narrow_ctas(int pieces) { return pieces == 1 ? 2 : 1; }

template <bool kF32>
__device__ __forceinline__ void ldg_res8(const void* base, size_t at, f32x2 (&a)[4]) {
  if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    pairs_of(__ldg(p), __ldg(p + 1), a);
  } else {
    unpack8(ld_stream_v4(static_cast<const uint16_t*>(base) + at), a);
  }
}

template <bool kF32, int kPieces, int kMode>
__global__ void __launch_bounds__(kNarrowThreads, narrow_ctas(kPieces))
    residual_norm_backward_narrow_kernel(const ResidualNormBackwardArgs a) {
  __shared__ __align__(16) float s_sum[kNarrowThreads / 32][kNarrowMaxH];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const GradHas has = grad_has<kMode>(a);
  const float inv_h = 1.0f / static_cast<float>(a.H);
  f32x2 gp[kPieces][4], gn[kPieces][4], acc_p[kPieces][4], acc_n[kPieces][4];
#pragma unroll
  for (int e = 0; e < kPieces; ++e)
    grad_weights(a, (lane + e * 32) * 8, (lane + e * 32) * 8 < a.H, gp[e], gn[e], acc_p[e],
                 acc_n[e]);
  const int step = gridDim.x * (kNarrowThreads / 32);
  for (int t = blockIdx.x * (kNarrowThreads / 32) + warp; t < a.T; t += step) {
    const float gt =
        a.gate_kind == kGateToken ? __ldg(static_cast<const float*>(a.gate) + t) : 1.f;
    f32x2 y[kPieces][4], v[kPieces][4], z[kPieces][4], d[kPieces][4], g[kPieces][4], q[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) q[i] = both(0.f);
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int col = (lane + e * 32) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[e][i] = v[e][i] = z[e][i] = d[e][i] = g[e][i] = both(0.f);
      if (col >= a.H) continue;
      const size_t at = static_cast<size_t>(t) * a.H + col;
      unpack8(ld_stream_v4(a.block + at), y[e]);
      ldg_res8<kF32>(a.residual_out, at, v[e]);
      if (has.next) unpack8(ld_stream_v4(a.grad_next + at), z[e]);
      if (has.dv) ldg_res8<kF32>(a.grad_residual_out, at, d[e]);
      if (has.full_gate) unpack8(ld_stream_v4(static_cast<const uint16_t*>(a.gate) + at), g[e]);
    }
#pragma unroll
    for (int e = 0; e < kPieces; ++e) grad_sums(q, has, y[e], v[e], z[e], d[e], g[e], gp[e], gn[e]);
    float sum[8] = {};
#pragma unroll
    for (int i = 0; i < 6; ++i) sum[i] = warp_sum_f(sum2(q[i]));
    const GradRow r = grad_row(sum, has, inv_h, a.eps, gt);
    if (a.gate_kind == kGateToken && lane == 0) static_cast<float*>(a.grad_gate)[t] = r.by;
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int col = (lane + e * 32) * 8;
      if (col >= a.H) continue;
      const size_t at = static_cast<size_t>(t) * a.H + col;
      grad_residual_piece(r, has, a.scale, v[e], z[e], d[e], gn[e], acc_n[e]);
      store_res8<kF32>(a.grad_residual, at, z[e]);
      grad_block_piece(r, has, inv_h, y[e], d[e], g[e], gp[e], acc_p[e]);
      if (has.full_gate)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.grad_gate) + at) = pack8(g[e]);
      *reinterpret_cast<uint4*>(a.grad_block + at) = pack8(d[e]);
    }
  }
  pdl_launch_dependents();
  const size_t plane = static_cast<size_t>(gridDim.x) * a.H;
  float* out = a.partials + static_cast<size_t>(blockIdx.x) * a.H;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (p == 0 ? !has.post && a.gate_kind != kGateChannel : !has.next) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
      if ((lane + e * 32) * 8 < a.H)
        store8(&s_sum[warp][(lane + e * 32) * 8], p == 0 ? acc_p[e] : acc_n[e]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += kNarrowThreads) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kNarrowThreads / 32; ++w) o += s_sum[w][c];
      out[p * plane + c] = o;
    }
  }
}

// After a wait that ran out: lets copies in flight land before the CTA exits, for limit_ns
// at most in all (a stage that nothing is on its way to keeps one parity open).
__device__ __noinline__ void drain_ring(uint64_t* full_bar, int stages, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  for (int i = 0; i < stages; ++i)
    for (uint32_t q = 0; q < 2; ++q)
      while (!mbar_try_wait(smem_u32(&full_bar[i]), q) && global_timer_ns() - t0 < limit_ns) {
      }
}

// After a wait that ran out, the ring kernels go on to the end of their rows for the
// barriers alone: nothing is fetched, and no value is stored that a row which did not come
// has entered. A thread learns of the others' waits with the row's sums: by the CTA's flag
// in the forward kernel, by the number of threads that gave up, summed with the rest, in
// the gradient's, whose CTAs may share rows.

// The forward pass for many rows and for rows wider than 8192, one to eight CTAs per SM:
// like the gradient's ring kernel below, kRows token rows at a time (adjacent in memory:
// one copy per array), which share the two barriers, kPieces 8-element pieces of each per
// thread.
template <bool kF32, int kThreads, int kRows, int kPieces>
__global__ void __launch_bounds__(kThreads, forward_ring_ctas(kThreads))
    residual_norm_ring_kernel(const ResidualNormArgs a, int stages, int stage_bytes,
                              uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full_bar[kRingMaxStages];
  __shared__ __align__(16) float red[2][kRows][32];
  __shared__ int abort_flag;
  static_assert(sizeof(full_bar) + sizeof(red) + 16 <= kForwardStatic, "resident_smem");
  volatile int* abort_v = &abort_flag;
  const int H = a.H;
  const uint32_t h2 = static_cast<uint32_t>(H) * 2, hr = kF32 ? h2 * 2 : h2;
  const bool has_post = a.post != nullptr, full_gate = a.gate_kind == kGateFull;
  const uint32_t at_x = kRows * h2, at_g = at_x + kRows * hr;  // arrays of a stage: y, x, gate
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full_bar[s]), 1);
    abort_flag = 0;
    mbar_fence_init();
  }
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(red) / 4); i += blockDim.x)
    (&red[0][0][0])[i] = 0.f;
  if constexpr (kThreads > kLateTriggerThreads) pdl_launch_dependents();
  pdl_wait();
  __syncthreads();

  auto fetch = [&](int t, int s) {  // one thread
    const uint32_t bar = smem_u32(&full_bar[s]);
    const uint32_t st = smem_u32(smem) + static_cast<uint32_t>(s) * stage_bytes;
    const uint32_t n = min(kRows, a.T - t);
    const size_t base = static_cast<size_t>(t) * H;
    mbar_arrive_expect_tx(bar, n * (h2 + hr + (full_gate ? h2 : 0)));
    bulk_load(st, a.block + base, n * h2, bar);
    bulk_load(st + at_x, static_cast<const uint8_t*>(a.residual) + base * (kF32 ? 4 : 2), n * hr,
              bar);
    if (full_gate) bulk_load(st + at_g, static_cast<const uint16_t*>(a.gate) + base, n * h2, bar);
  };
  const int step = gridDim.x * kRows, begin = blockIdx.x * kRows;
  const int64_t copied = min(static_cast<int64_t>(a.T), a.ring.copied);
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) {
      const int64_t t = begin + static_cast<int64_t>(s) * step;
      if (t < copied) fetch(static_cast<int>(t), s);
    }

  // Post weight (times a channel gate), next weight. With two pieces and more than 640
  // threads the next weight is loaded for each row instead of held (T = 3500: H = 16384
  // 74 us, 83 when held, with spills; H = 11520 54.7 and 58.5).
  constexpr bool kHoldNext = kPieces == 1 || kThreads <= 640;
  f32x2 gp[kPieces][4], gn[kPieces][4];
#pragma unroll
  for (int e = 0; e < kPieces; ++e) {
    const int col = (threadIdx.x + e * blockDim.x) * 8;
    const bool on = col < H;
#pragma unroll
    for (int i = 0; i < 4; ++i) gp[e][i] = both(1.f), gn[e][i] = both(0.f);
    if (on && has_post) load8(a.post + col, gp[e]);
    if (kHoldNext && on && a.next != nullptr) load8(a.next + col, gn[e]);
    if (on && a.gate_kind == kGateChannel) {
      f32x2 g[4];
      load8(static_cast<const float*>(a.gate) + col, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) gp[e][i] = mul2(gp[e][i], g[i]);
    }
  }
  const float inv_h = 1.0f / static_cast<float>(H);
  const f32x2 scale = both(a.scale);
  int s = 0, turn = 0;
  uint32_t parity = 0;
  bool ok = true;
  for (int t = begin; t < a.T; t += step) {
    const uint8_t* st = smem + static_cast<size_t>(s) * stage_bytes;
    if (ok) ok = mbar_wait(smem_u32(&full_bar[s]), parity, err, abort_v, a.ring.limit_ns);
    float sum[kRows], factor[kRows];  // of y: r1 and a token gate
    uint4 y_raw[kRows][kPieces];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      factor[r] = a.gate_kind == kGateToken && t + r < a.T
                      ? __ldg(static_cast<const float*>(a.gate) + t + r)
                      : 1.f;
      f32x2 q = both(0.f);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int lane = threadIdx.x + e * blockDim.x;  // piece of the row
        f32x2 f[4];
        y_raw[r][e] = make_uint4(0, 0, 0, 0);
        if (lane * 8 < H && t + r < a.T)
          y_raw[r][e] = *reinterpret_cast<const uint4*>(st + r * h2 + lane * 16);
        unpack8(y_raw[r][e], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(f[i], f[i], q);
      }
      sum[r] = sum2(q);
    }
    if (has_post) {
      if (!cta_sum<kRows, 1>(sum, red[turn], abort_v)) ok = false;
      turn ^= 1;
#pragma unroll
      for (int r = 0; r < kRows; ++r) factor[r] *= 1.0f / sqrtf(sum[r] * inv_h + a.eps);
    }
    f32x2 v[kRows][kPieces][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      f32x2 q = both(0.f);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int lane = threadIdx.x + e * blockDim.x, col = lane * 8;
        if (col >= H || t + r >= a.T) continue;
        f32x2 f[4];
        const f32x2 c = both(factor[r]);
        unpack8(y_raw[r][e], f);
        lds_res8<kF32>(st + at_x + r * hr, lane, v[r][e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], c), gp[e][i]);
        if (full_gate) {
          f32x2 g[4];
          lds8(st + at_g + r * h2, lane, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], g[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[r][e][i] = fma2(scale, v[r][e][i], f[i]);
          q = fma2(v[r][e][i], v[r][e][i], q);
        }
        if (ok) store_res8<kF32>(a.residual_out, static_cast<size_t>(t + r) * H + col, v[r][e]);
      }
      sum[r] = sum2(q);
    }
    // Also without a second norm: after this barrier all threads are done with the stage.
    if (!cta_sum<kRows, 1>(sum, red[turn], abort_v)) ok = false;
    turn ^= 1;
    if (a.next != nullptr && ok) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const f32x2 r2 = both(1.0f / sqrtf(sum[r] * inv_h + a.eps));
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
          const int col = (threadIdx.x + e * blockDim.x) * 8;
          if (col >= H || t + r >= a.T) continue;
          f32x2 o[4];
          if constexpr (!kHoldNext) load8(a.next + col, gn[e]);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul2(mul2(v[r][e][i], r2), gn[e][i]);
          *reinterpret_cast<uint4*>(a.next_out + static_cast<size_t>(t + r) * H + col) = pack8(o);
        }
      }
    }
    // Refilled after the row's stores: asking for it right after the barrier measured
    // 1-4 % slower.
    if (threadIdx.x == 0 && ok && t + static_cast<int64_t>(stages) * step < copied)
      fetch(t + stages * step, s);
    if (++s == stages) s = 0, parity ^= 1;
  }
  if constexpr (kThreads <= kLateTriggerThreads) pdl_launch_dependents();
  if (threadIdx.x == 0 && !ok) drain_ring(full_bar, stages, a.ring.limit_ns);
}

template <bool kF32, int kThreads, int kPieces, int kMode, int kCluster>
__global__ void __launch_bounds__(kThreads, kPieces == 2 ? 1 : ring_ctas_per_sm(kThreads))
    residual_norm_backward_ring_kernel(const ResidualNormBackwardArgs a, int stages,
                                       int stage_bytes, uint32_t* err) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full_bar[kRingMaxStages];
  __shared__ __align__(16) float red[2][8][32];
  __shared__ int abort_flag;
  static_assert(sizeof(full_bar) + sizeof(red) + 16 <= kBackwardStatic, "resident_smem");
  volatile int* abort_v = &abort_flag;
  static_assert(kCluster == 1 || kThreads <= 512, "half a plane of `red` per CTA");
  const int H = a.H;
  const RowPart part = row_part<kCluster>(H);
  const uint32_t h2 = static_cast<uint32_t>(part.width) * 2, hr = kF32 ? h2 * 2 : h2;
  const GradHas has = grad_has<kMode>(a);
  const bool has_post = has.post, has_next = has.next, has_dv = has.dv, full_gate = has.full_gate;
  // Arrays of a stage: y, v, dz, dv, gate.
  const uint32_t at_v = h2, at_z = at_v + hr, at_d = at_z + (has_next ? h2 : 0),
                 at_g = at_d + (has_dv ? hr : 0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full_bar[s]), 1);
    abort_flag = 0;
    mbar_fence_init();
  }
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(red) / 4); i += blockDim.x)
    (&red[0][0][0])[i] = 0.f;
  pdl_wait();
  if constexpr (kCluster == 1)
    __syncthreads();
  else
    cluster_sync();  // the other CTA's `red` is zeroed too

  auto fetch = [&](int t, int s) {  // one thread
    const uint32_t bar = smem_u32(&full_bar[s]);
    const uint32_t st = smem_u32(smem) + static_cast<uint32_t>(s) * stage_bytes;
    const size_t base = static_cast<size_t>(t) * H + part.first;
    const size_t rb = base * (kF32 ? 4 : 2);
    mbar_arrive_expect_tx(bar, at_g + (full_gate ? h2 : 0));
    bulk_load(st, a.block + base, h2, bar);
    bulk_load(st + at_v, static_cast<const uint8_t*>(a.residual_out) + rb, hr, bar);
    if (has_next) bulk_load(st + at_z, a.grad_next + base, h2, bar);
    if (has_dv) bulk_load(st + at_d, static_cast<const uint8_t*>(a.grad_residual_out) + rb, hr, bar);
    if (full_gate) bulk_load(st + at_g, static_cast<const uint16_t*>(a.gate) + base, h2, bar);
  };
  const int step = gridDim.x / kCluster, begin = blockIdx.x / kCluster;
  const int64_t copied = min(static_cast<int64_t>(a.T), a.ring.copied);
  if (threadIdx.x == 0)
    for (int s = 0; s < stages && begin + s * step < copied; ++s) fetch(begin + s * step, s);

  f32x2 gp[kPieces][4], gn[kPieces][4], acc_p[kPieces][4], acc_n[kPieces][4];
#pragma unroll
  for (int e = 0; e < kPieces; ++e)
    grad_weights(a, part.first + (threadIdx.x + e * blockDim.x) * 8,
                 static_cast<int>(threadIdx.x + e * blockDim.x) * 8 < part.width, gp[e], gn[e],
                 acc_p[e], acc_n[e]);
  const float inv_h = 1.0f / static_cast<float>(H);
  int s = 0, turn = 0, last = -1;  // last: the row before
  uint32_t parity = 0;
  bool ok = true;
  for (int t = begin; t < a.T; t += step) {
    const uint8_t* st = smem + static_cast<size_t>(s) * stage_bytes;
    const float gt =
        a.gate_kind == kGateToken ? __ldg(static_cast<const float*>(a.gate) + t) : 1.f;
    if (ok) ok = mbar_wait(smem_u32(&full_bar[s]), parity, err, abort_v, a.ring.limit_ns);
    float sum[8] = {};
    f32x2 q[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) q[i] = both(0.f);
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int lane = threadIdx.x + e * blockDim.x;  // piece of the row
      if (lane * 8 >= part.width) continue;
      f32x2 y[4], v[4], z[4], d[4], g[4];
      lds8(st, lane, y);
      lds_res8<kF32>(st + at_v, lane, v);
      if (has_next) lds8(st + at_z, lane, z);
      if (has_dv) lds_res8<kF32>(st + at_d, lane, d);
      if (full_gate) lds8(st + at_g, lane, g);
      grad_sums(q, has, y, v, z, d, g, gp[e], gn[e]);
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) sum[i] = sum2(q[i]);
    sum[6] = ok ? 0.f : 1.f;  // threads that gave up, in both CTAs of a cluster
    cta_sum<8, kCluster>(sum, red[turn]);
    turn ^= 1;
    ok = sum[6] == 0.f;
    if (!ok) continue;
    // All threads are done with the previous row's stage.
    if (threadIdx.x == 0 && last >= 0 && last + static_cast<int64_t>(stages) * step < copied)
      fetch(last + stages * step, s == 0 ? stages - 1 : s - 1);
    last = t;
    const GradRow r = grad_row(sum, has, inv_h, a.eps, gt);
    if (a.gate_kind == kGateToken && threadIdx.x == 0 && part.first == 0)
      static_cast<float*>(a.grad_gate)[t] = r.by;
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int lane = threadIdx.x + e * blockDim.x;
      if (lane * 8 >= part.width) continue;
      const size_t base = static_cast<size_t>(t) * H + part.first + lane * 8;
      f32x2 y[4], v[4], z[4], d[4], g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = d[i] = both(0.f);
      if (has_dv) lds_res8<kF32>(st + at_d, lane, d);
      if (has_next) {
        lds_res8<kF32>(st + at_v, lane, v);
        lds8(st + at_z, lane, z);
      }
      grad_residual_piece(r, has, a.scale, v, z, d, gn[e], acc_n[e]);
      store_res8<kF32>(a.grad_residual, base, z);
      lds8(st, lane, y);
      if (full_gate) lds8(st + at_g, lane, g);
      grad_block_piece(r, has, inv_h, y, d, g, gp[e], acc_p[e]);
      if (full_gate)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.grad_gate) + base) = pack8(g);
      *reinterpret_cast<uint4*>(a.grad_block + base) = pack8(d);
    }
    if (++s == stages) s = 0, parity ^= 1;
  }
  // Not before: CTAs of the next kernel would take the places of this one's that are
  // not resident yet (measured: 52 against 38 us at T = 4614, H = 1224, FP32).
  pdl_launch_dependents();
  const size_t plane = static_cast<size_t>(step) * H;
#pragma unroll
  for (int e = 0; e < kPieces; ++e) {
    const int col = (threadIdx.x + e * blockDim.x) * 8;
    if (col >= part.width) continue;
    const size_t at = static_cast<size_t>(begin) * H + part.first + col;
    if (has_post || a.gate_kind == kGateChannel) store8(a.partials + at, acc_p[e]);
    if (has_next) store8(a.partials + plane + at, acc_n[e]);
  }
  if (threadIdx.x == 0 && !ok) drain_ring(full_bar, stages, a.ring.limit_ns);
}

struct RingPlan {
  int stages = 0, stage_bytes = 0, threads = 0, rows = 1;
  size_t smem = 0;
};

// The forward ring; stages == 0 when the direct kernel takes the call.
RingPlan ring_plan(const ResidualNormArgs& a, int num_sms) {
  RingPlan r;
  if (a.H < kForwardRingMinH || (a.H <= kRingMaxH && a.T < kRingMinRowsPerSm * num_sms)) return r;
  const int halves = 1 + (a.residual_f32 ? 2 : 1) + (a.gate_kind == kGateFull ? 1 : 0);
  r.rows = forward_ring_rows(a.H, halves);
  r.stage_bytes = forward_stage_bytes(a.H, halves, r.rows);
  r.threads = forward_ring_threads(a.H);
  r.stages = forward_ring_stages(a.H, r.stage_bytes);
  r.smem = static_cast<size_t>(r.stages) * r.stage_bytes;
  return r;
}

// The gradient's ring; stages == 0 for narrow rows.
RingPlan ring_plan(const ResidualNormBackwardArgs& a) {
  RingPlan r;
  if (a.H < kRingMinH) return r;
  const int width = ring_width(a.H);
  const int h2 = width * 2, hr = a.residual_f32 ? h2 * 2 : h2;
  const int bytes = h2 + hr + (a.next != nullptr ? h2 : 0) +
                    (a.grad_residual_out != nullptr ? hr : 0) +
                    (a.gate_kind == kGateFull ? h2 : 0);
  r.stage_bytes = (bytes + 127) / 128 * 128;
  r.threads = backward_ring_threads(width);
  r.stages = backward_ring_stages(width, r.stage_bytes);
  r.smem = static_cast<size_t>(r.stages) * r.stage_bytes;
  return r;
}

// Sums of the partial rows, in a fixed order: a CTA's threads take slices of the rows of
// its columns, then a tree adds the slices. Plane 0 gives the gradients of the post weight
// and of a channel gate, plane 1 that of the next weight.
template <int kReduceCols>
__global__ void __launch_bounds__(kReduceThreads)
    column_sum_kernel(const float* __restrict__ partials, const float* __restrict__ post,
                      const float* __restrict__ gate, float* __restrict__ grad_post,
                      float* __restrict__ grad_gate, float* __restrict__ grad_next,
                      int partial_rows, int H) {
  constexpr int kReduceSlices = kReduceThreads / kReduceCols;
  __shared__ float4 s_part[kReduceSlices][kReduceCols];
  pdl_wait();
  if (blockIdx.y == 0 ? grad_post == nullptr && grad_gate == nullptr : grad_next == nullptr) return;
  const int cx = threadIdx.x % kReduceCols, slice = threadIdx.x / kReduceCols;
  const int col = (blockIdx.x * kReduceCols + cx) * 4;
  const float* src = partials + blockIdx.y * static_cast<size_t>(partial_rows) * H + col;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H) {
#pragma unroll 8
    for (int r = slice; r < partial_rows; r += kReduceSlices) {
      const float4 v = *reinterpret_cast<const float4*>(src + static_cast<size_t>(r) * H);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  pdl_launch_dependents();
  s_part[slice][cx] = s;
#pragma unroll
  for (int n = kReduceSlices / 2; n > 0; n /= 2) {
    __syncthreads();
    if (slice < n) {
      const float4 v = s_part[slice + n][cx];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      s_part[slice][cx] = s;
    }
  }
  if (slice != 0 || col >= H) return;
  if (blockIdx.y == 1) {
    *reinterpret_cast<float4*>(grad_next + col) = s;
    return;
  }
  auto times = [&](const float* f) {
    const float4 w = f == nullptr ? make_float4(1.f, 1.f, 1.f, 1.f)
                                  : *reinterpret_cast<const float4*>(f + col);
    return make_float4(s.x * w.x, s.y * w.y, s.z * w.z, s.w * w.w);
  };
  if (grad_post != nullptr) *reinterpret_cast<float4*>(grad_post + col) = times(gate);
  if (grad_gate != nullptr) *reinterpret_cast<float4*>(grad_gate + col) = times(post);
}

// Rows that the backward kernels work on at once (with all their CTAs resident), and so
// the rows of partial sums: CTAs, or clusters of two. (T = 8192, H = 512 17.6 us, 19.4 with
// twice the CTAs that an SM holds; T = 2500, H = 384 7.5 and 9.1.)
int backward_rows(int T, int H, int num_sms) {
  if (H > kNarrowMaxH)
    return std::min(T, num_sms * backward_ring_ctas(ring_width(H)) / ring_cluster(H));
  const int rows = kNarrowThreads / 32;
  return std::min((T + rows - 1) / rows, narrow_ctas(H <= 256 ? 1 : 2) * num_sms);
}

}  // namespace

int residual_norm_partial_rows(int T, int H) {
  return backward_rows(T, H, kMaxSms);
}

namespace {

typedef void (*ForwardRingKernel)(const ResidualNormArgs, int, int, uint32_t*);
typedef void (*RingKernel)(const ResidualNormBackwardArgs, int, int, uint32_t*);

typedef void (*NarrowKernel)(const ResidualNormBackwardArgs);

template <int kMode>
NarrowKernel narrow_kernel(int H, bool f32) {
  if (H <= 256)
    return f32 ? residual_norm_backward_narrow_kernel<true, 1, kMode>
               : residual_norm_backward_narrow_kernel<false, 1, kMode>;
  return f32 ? residual_norm_backward_narrow_kernel<true, 2, kMode>
             : residual_norm_backward_narrow_kernel<false, 2, kMode>;
}

NarrowKernel narrow_kernel(int H, bool f32, int mode) {
  return mode == kSome  ? narrow_kernel<kSome>(H, f32)
         : mode == kAll ? narrow_kernel<kAll>(H, f32)
                        : narrow_kernel<kAllGated>(H, f32);
}

template <int kRows, int kPieces>
ForwardRingKernel forward_ring_kernel(int threads, bool f32) {
  if constexpr (kPieces == 1) {
    if (threads <= 96)
      return f32 ? residual_norm_ring_kernel<true, 96, kRows, kPieces>
                 : residual_norm_ring_kernel<false, 96, kRows, kPieces>;
    if (threads <= 128)
      return f32 ? residual_norm_ring_kernel<true, 128, kRows, kPieces>
                 : residual_norm_ring_kernel<false, 128, kRows, kPieces>;
    if (threads <= 288)
      return f32 ? residual_norm_ring_kernel<true, 288, kRows, kPieces>
                 : residual_norm_ring_kernel<false, 288, kRows, kPieces>;
    if (threads <= 448)
      return f32 ? residual_norm_ring_kernel<true, 448, kRows, kPieces>
                 : residual_norm_ring_kernel<false, 448, kRows, kPieces>;
  }
  if (threads <= 640)
    return f32 ? residual_norm_ring_kernel<true, 640, kRows, kPieces>
               : residual_norm_ring_kernel<false, 640, kRows, kPieces>;
  if (threads <= 896)
    return f32 ? residual_norm_ring_kernel<true, 896, kRows, kPieces>
               : residual_norm_ring_kernel<false, 896, kRows, kPieces>;
  return f32 ? residual_norm_ring_kernel<true, 1024, kRows, kPieces>
             : residual_norm_ring_kernel<false, 1024, kRows, kPieces>;
}

ForwardRingKernel forward_ring_kernel(int H, int rows, int threads, bool f32) {
  if (H > kRingMaxH) return forward_ring_kernel<1, 2>(threads, f32);
  if (rows == 2) return forward_ring_kernel<2, 1>(threads, f32);
  return threads <= 448 ? residual_norm_ring_kernel<true, 448, 1, 1>  // (single_rows_as_built)
                        : residual_norm_ring_kernel<true, 1024, 1, 1>;
}

template <bool kF32>
auto forward_kernel(const Shape& s) -> void (*)(const ResidualNormArgs, int) {
  return s.pieces == 1 ? residual_norm_kernel<1, kF32> : residual_norm_kernel<2, kF32>;
}

template <bool kF32, int kMode>
RingKernel ring_kernel(int H) {
  const int width = ring_width(H), threads = backward_ring_threads(width);
  if (ring_cluster(H) == 2)
    return threads <= 448 ? residual_norm_backward_ring_kernel<kF32, 448, 2, kMode, 2>
                          : residual_norm_backward_ring_kernel<kF32, 512, 2, kMode, 2>;
  if (threads <= 128) return residual_norm_backward_ring_kernel<kF32, 128, 1, kMode, 1>;
  if (backward_ring_pieces(width) == 1)
    return threads <= 288 ? residual_norm_backward_ring_kernel<kF32, 288, 1, kMode, 1>
                          : residual_norm_backward_ring_kernel<kF32, 448, 1, kMode, 1>;
  return threads <= 448 ? residual_norm_backward_ring_kernel<kF32, 448, 2, kMode, 1>
                        : residual_norm_backward_ring_kernel<kF32, 512, 2, kMode, 1>;
}

RingKernel ring_kernel(int H, bool f32, int mode) {
  switch (mode) {
    case kSome: return f32 ? ring_kernel<true, kSome>(H) : ring_kernel<false, kSome>(H);
    case kAll: return f32 ? ring_kernel<true, kAll>(H) : ring_kernel<false, kAll>(H);
    default: return f32 ? ring_kernel<true, kAllGated>(H) : ring_kernel<false, kAllGated>(H);
  }
}

}  // namespace

cudaError_t setup_residual_norm(const DeviceInfo&) {
  for (bool f32 : {false, true}) {
    cudaError_t e;
    for (int H : {4096, 16384})
      for (int rows : {1, 2})
        for (int threads : {96, 128, 288, 448, 640, 896, 1024})
          if ((e = cudaFuncSetAttribute(forward_ring_kernel(H, rows, threads, f32),
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kRingSmem))) != cudaSuccess)
            return e;
    for (int H : {1024, 2304, 3584, 7168, 8192, 14336, 16384})  // one of each kernel
      for (int mode : {kSome, kAll, kAllGated})
        if ((e = cudaFuncSetAttribute(ring_kernel(H, f32, mode),
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(backward_ring_smem(ring_width(H))))) !=
            cudaSuccess)
          return e;
  }
  return cudaSuccess;
}

cudaError_t launch_residual_norm(const ResidualNormArgs& a, const DeviceInfo& dev,
                                 cudaStream_t stream) {
  const RingPlan ring = ring_plan(a, dev.num_sms);
  if (ring.stages != 0)
    return launch_dependent(forward_ring_kernel(a.H, ring.rows, ring.threads, a.residual_f32),
                            dim3(std::min((a.T + ring.rows - 1) / ring.rows,
                                          dev.num_sms * forward_ring_ctas(ring.threads))),
                            dim3(ring.threads), ring.smem, stream, a, ring.stages,
                            ring.stage_bytes, dev.err_word);
  const Shape s = shape_of(a.H);
  const dim3 grid((a.T + s.per_cta - 1) / s.per_cta);
  return launch_dependent(a.residual_f32 ? forward_kernel<true>(s) : forward_kernel<false>(s), grid,
                          dim3(s.threads), 0, stream, a, s.tpr);
}

cudaError_t launch_residual_norm_backward(const ResidualNormBackwardArgs& a,
                                          const DeviceInfo& dev, cudaStream_t stream) {
  const int rows = backward_rows(a.T, a.H, std::min(dev.num_sms, kMaxSms));
  cudaError_t e;
  if (a.H <= kNarrowMaxH) {
    e = launch_dependent(narrow_kernel(a.H, a.residual_f32, grad_mode(a)), dim3(rows),
                         dim3(kNarrowThreads), 0, stream, a);
  } else {
    const RingPlan ring = ring_plan(a);
    const int cluster = ring_cluster(a.H);
    e = launch_dependent_clusters(cluster, ring_kernel(a.H, a.residual_f32, grad_mode(a)),
                                  dim3(rows * cluster), dim3(ring.threads), ring.smem, stream, a,
                                  ring.stages, ring.stage_bytes, dev.err_word);
  }
  const bool channel = a.gate_kind == kGateChannel;
  if (e != cudaSuccess || (a.post == nullptr && a.next == nullptr && !channel)) return e;
  const int cols = a.H <= kReduceNarrowH ? 4 : 16;
  return launch_dependent(cols == 4 ? column_sum_kernel<4> : column_sum_kernel<16>,
                          dim3((a.H / 4 + cols - 1) / cols, 2), dim3(kReduceThreads), 0, stream,
                          static_cast<const float*>(a.partials), a.post,
                          channel ? static_cast<const float*>(a.gate) : nullptr, a.grad_post,
                          channel ? static_cast<float*>(a.grad_gate) : nullptr,
                          a.grad_next_weight, rows, a.H);
}

}  // namespace lt
