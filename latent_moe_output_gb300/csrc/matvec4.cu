// latent_tail_expert_matvec4: products of expert-sorted rows with 4-bit weights
// that carry one scale per group of G columns.
//
//   out[r,m] = sum_c x[r,c] * (q[e,m,c] - 8) * s[e,m,c/G]
//            = sum_groups s[e,m,g] * ( sum_{c in g} x[r,c] * (q[e,m,c] - 8) )
//
// With the few rows per expert of a decode step the weights are read once and
// used at most a few times, so their stream bounds the call; the work per weight
// is the unpacking. A 4-bit value plus 128 is one bit operation away from a bf16
// number (0x4300 | q = 128 + q), and 136 less is exactly q - 8, so the inner sums
// run on the tensor cores with exact bf16 operands and FP32 accumulators: 16 weight
// rows x 16 columns against 8 rows of x per instruction. These warp-level
// instructions take their operands from registers, where the unpacked weights are;
// the tcgen05 ones would need them written back to shared memory first, and at 8
// to 32 rows the tensor rate does not matter. Scales multiply the FP32 group sums.
//
// Layout of the work. A tile is kRows = 128 / kSplit weight rows of one expert,
// against up to 8 * kTiles rows of x (a pass). The CTAs walk over the tiles of
// the experts that have rows (found from the offsets at the start of the kernel).
// One warp streams weights and x through a ring of stages with TMA: a stage holds
// kSplit boxes of 256 columns (kRows x 128 bytes of weights, swizzled so that the
// eight rows of a fragment lie in different banks, and 8 * kTiles rows of x). The
// eight other warps each own 16 weight rows and one of the kSplit column parts of
// every stage; the parts are added in order through shared memory at the end of a
// tile. kSplit = 4 gives enough tiles to fill the GPU from one matrix.
#include "block_launch.h"
#include "rows.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kConsumers = 8;  // warps
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kBoxCols = 256;  // columns per box: 128 bytes of weights
constexpr int kMaxStages = 8;
constexpr int kSmemBudget = 102 * 1024;  // dynamic, two CTAs per SM

template <int kSplit, int kTiles>
struct Config {
  static constexpr int kRows = 128 / kSplit;
  static constexpr int kWeightBytes = 128 * 128;
  static constexpr int kXBoxBytes = 8 * 128;  // 8 rows x 64 columns
  static constexpr int kStageBytes = kWeightBytes + kSplit * kTiles * 4 * kXBoxBytes;
  // Column parts 1.. of a tile's sums, double-buffered.
  static constexpr int kSumFloats = (kSplit - 1) * kRows * 8 * kTiles;
  static constexpr int kSumBytes = 2 * kSumFloats * 4;
  static constexpr int kStages =
      (kSmemBudget - kSumBytes - 1024) / kStageBytes > kMaxStages
          ? kMaxStages
          : (kSmemBudget - kSumBytes - 1024) / kStageBytes;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + kSumBytes + 1024;
  static_assert(kStages >= 2, "a ring needs two stages");
};

struct Params {
  const uint16_t* scales;
  const int32_t* offsets;
  uint16_t* out;
  int N, E, M, C;
  uint32_t* err;
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

// Values i and i + 4 of the eight in w, minus 8, as two bf16 numbers (exact).
__device__ __forceinline__ uint32_t weight_pair(uint32_t w, int i) {
  const uint32_t biased = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;  // 128 + q
  uint32_t v;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(biased), "r"(0x43084308u));  // - 136
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void consumer_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

// Rows [row0, row0 + rows) of expert e against weight rows m0...
struct Tile {
  int e, row0, rows, m0;
};

__device__ __forceinline__ Tile tile_at(int64_t tile, int mblocks, int rows_per_tile,
                                        int rows_per_pass, const int* s_first,
                                        const int* s_unit, int E) {
  const int unit = static_cast<int>(tile / mblocks);
  int lo = 0, hi = E - 1;  // the expert with s_unit[e] <= unit < s_unit[e + 1]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s_unit[mid + 1] > unit)
      hi = mid;
    else
      lo = mid + 1;
  }
  Tile t;
  t.e = lo;
  t.row0 = s_first[lo] + (unit - s_unit[lo]) * rows_per_pass;
  t.rows = min(rows_per_pass, s_first[lo + 1] - t.row0);
  t.m0 = static_cast<int>(tile % mblocks) * rows_per_tile;
  return t;
}

template <int kGroup, int kSplit, int kTiles>
__global__ void __launch_bounds__(kThreads, 2)
    matvec4_kernel(const __grid_constant__ CUtensorMap w_map,
                   const __grid_constant__ CUtensorMap x_map, const Params p) {
  using Cfg = Config<kSplit, kTiles>;
  constexpr int kPass = 8 * kTiles;
  constexpr int kScales = kBoxCols / kGroup;  // per row and box
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[Cfg::kStages], empty_bar[Cfg::kStages];
  __shared__ int s_first[kMaxExperts + 1];  // first row of each expert
  __shared__ int s_unit[kMaxExperts + 1];   // passes before each expert
  __shared__ int abort_flag;
  volatile int* abort_v = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), kConsumers);
    }
    abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&w_map);
    tma_prefetch_map(&x_map);
  }
  pdl_launch_dependents();
  pdl_wait();
  if (p.offsets != nullptr) {
    for (int e = threadIdx.x; e <= p.E; e += kThreads)
      s_first[e] = min(max(p.offsets[e], 0), p.N);
  } else if (threadIdx.x == 0) {
    s_first[0] = 0;
    s_first[1] = p.N;
  }
  __syncthreads();
  if (warp == 0) {
    // Running maximum (offsets that run backwards give empty experts) and the
    // exclusive sum of the passes; each lane takes a contiguous part.
    const int per = (p.E + 32) / 32;
    const int lo = min(p.E + 1, lane * per), hi = min(p.E + 1, lo + per);
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
    __syncwarp();
    int sum = 0;
    for (int e = lo; e < hi && e < p.E; ++e) sum += (s_first[e + 1] - s_first[e] + kPass - 1) / kPass;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    run = incl - sum;
    for (int e = lo; e < hi; ++e) {
      s_unit[e] = run;
      if (e < p.E) run += (s_first[e + 1] - s_first[e] + kPass - 1) / kPass;
    }
  }
  __syncthreads();

  const int mblocks = (p.M + Cfg::kRows - 1) / Cfg::kRows;
  const int64_t tiles = static_cast<int64_t>(s_unit[p.E]) * mblocks;
  const int boxes = (p.C + kBoxCols - 1) / kBoxCols;
  const int steps = (boxes + kSplit - 1) / kSplit;  // stages per tile

  if (warp == kConsumers) {
    if (lane == 0) {
      uint32_t it = 0;  // stages issued
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const Tile t = tile_at(tile, mblocks, Cfg::kRows, kPass, s_first, s_unit, p.E);
        const int n_tiles = (t.rows + 7) / 8;
        for (int i = 0; i < steps; ++i, ++it) {
          const uint32_t s = it % Cfg::kStages;
          ok = mbar_wait(smem_u32(&empty_bar[s]), ((it / Cfg::kStages) & 1u) ^ 1u, p.err, abort_v);
          if (!ok) break;
          const int live = min(kSplit, boxes - i * kSplit);
          const uint32_t bar = smem_u32(&full_bar[s]);
          const uint32_t st = ring + s * Cfg::kStageBytes;
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live) *
                                         (Cfg::kRows * 128 + n_tiles * 4 * Cfg::kXBoxBytes));
          for (int j = 0; j < live; ++j) {
            const int c0 = (i * kSplit + j) * kBoxCols;
            tma_load_2d(st + j * Cfg::kRows * 128, &w_map, bar, c0 / 2, t.e * p.M + t.m0);
            const uint32_t xs = st + Cfg::kWeightBytes + j * kTiles * 4 * Cfg::kXBoxBytes;
            for (int n = 0; n < n_tiles; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                tma_load_2d(xs + (n * 4 + c) * Cfg::kXBoxBytes, &x_map, bar, c0 + c * 64,
                            t.row0 + n * 8);
          }
        }
      }
      if (!ok) {  // let copies already in flight land before the CTA exits
        for (uint32_t i = it > Cfg::kStages ? it - Cfg::kStages : 0; i < it; ++i) {
          const uint32_t bar = smem_u32(&full_bar[i % Cfg::kStages]);
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(bar, (i / Cfg::kStages) & 1u) &&
                 global_timer_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else {
    const int part = warp / (kConsumers / kSplit);       // column part of every stage
    const int mrow = warp % (kConsumers / kSplit) * 16;  // first weight row in the tile
    const int g = lane >> 2, c4 = lane & 3;
    // Column n of a fragment holds row (n >> 1) + 4 (n & 1) of the eight: lanes of
    // one quarter of the warp then read different halves of the swizzled rows.
    const int xrow = (g >> 1) + (g & 1) * 4;
    float* sums = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) +
                                           Cfg::kStages * Cfg::kStageBytes);
    const int pitch = p.C / kGroup;  // scales per row
    const bool vec = pitch % kScales == 0;
    uint32_t it = 0;
    bool ok = true;
    int parity = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const Tile t = tile_at(tile, mblocks, Cfg::kRows, kPass, s_first, s_unit, p.E);
      const int n_tiles = (t.rows + 7) / 8;
      const uint16_t* srow[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)  // (rows past the matrix are read from its last row)
        srow[h] = p.scales + (static_cast<size_t>(t.e) * p.M +
                              min(p.M - 1, t.m0 + mrow + g + h * 8)) * pitch;
      // Scales of one box: kScales per row, two per register.
      auto load_scales = [&](int box, uint32_t (&sc)[2][kScales / 2]) {
        const int first = box * kScales;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (vec) {
            if (first < pitch) {
              if constexpr (kScales == 8) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(srow[h] + first));
                sc[h][0] = v.x; sc[h][1] = v.y; sc[h][2] = v.z; sc[h][3] = v.w;
              } else if constexpr (kScales == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(srow[h] + first));
                sc[h][0] = v.x; sc[h][1] = v.y;
              } else {
                sc[h][0] = __ldg(reinterpret_cast<const uint32_t*>(srow[h] + first));
              }
            }
          } else {
#pragma unroll
            for (int q = 0; q < kScales / 2; ++q) {
              const uint32_t a = first + 2 * q < pitch ? __ldg(srow[h] + first + 2 * q) : 0;
              const uint32_t b = first + 2 * q + 1 < pitch ? __ldg(srow[h] + first + 2 * q + 1) : 0;
              sc[h][q] = a | (b << 16);
            }
          }
        }
      };
      float total[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[n][j] = 0.f;

      uint32_t next[2][kScales / 2] = {};
      load_scales(part, next);
      for (int i = 0; i < steps; ++i, ++it) {
        uint32_t sc[2][kScales / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < kScales / 2; ++q) sc[h][q] = next[h][q];
        if (i + 1 < steps) load_scales((i + 1) * kSplit + part, next);
        const uint32_t s = it % Cfg::kStages;
        if (ok) ok = mbar_wait(smem_u32(&full_bar[s]), (it / Cfg::kStages) & 1u, p.err, abort_v);
        const int box = i * kSplit + part;
        if (ok && box < boxes) {
          const uint32_t st = ring + s * Cfg::kStageBytes;
          const uint32_t wa = st + part * Cfg::kRows * 128 + (mrow + g) * 128 + c4 * 4;
          const uint32_t xa = st + Cfg::kWeightBytes + part * kTiles * 4 * Cfg::kXBoxBytes +
                              xrow * 128;
          const int runs = min(8, (p.C - box * kBoxCols) / 32);  // runs of 32 columns
          float acc[kTiles][4];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j >= runs) break;
            constexpr int kRunsPerGroup = kGroup / 32;
            const uint32_t w0 = lds32(wa + ((j ^ g) << 4));
            const uint32_t w1 = lds32(wa + 8 * 128 + ((j ^ g) << 4));
            uint32_t a0[4], a1[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              a0[q] = weight_pair(w0, q);
              a1[q] = weight_pair(w1, q);
            }
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
              if (n >= n_tiles) break;
              if (j % kRunsPerGroup == 0) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
              const uint4 v = lds128(xa + (n * 4 + (j >> 1)) * Cfg::kXBoxBytes +
                                     ((((j & 1) * 4 + c4) ^ xrow) << 4));
              mma_bf16(acc[n], a0[0], a1[0], a0[1], a1[1], __byte_perm(v.x, v.z, 0x5410),
                       __byte_perm(v.x, v.z, 0x7632));
              mma_bf16(acc[n], a0[2], a1[2], a0[3], a1[3], __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
              if (j % kRunsPerGroup == kRunsPerGroup - 1) {
                constexpr int kShift = kRunsPerGroup;
                const int q = j / kShift;
                const float s0 = (q & 1) ? bf16_hi(sc[0][q >> 1]) : bf16_lo(sc[0][q >> 1]);
                const float s1 = (q & 1) ? bf16_hi(sc[1][q >> 1]) : bf16_lo(sc[1][q >> 1]);
                total[n][0] = fmaf(s0, acc[n][0], total[n][0]);
                total[n][1] = fmaf(s0, acc[n][1], total[n][1]);
                total[n][2] = fmaf(s1, acc[n][2], total[n][2]);
                total[n][3] = fmaf(s1, acc[n][3], total[n][3]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty_bar[s]));
      }

      // Element (j, lane) of a fragment: weight row g + 8 (j >> 1), column
      // 2 c4 + (j & 1), i.e. row c4 + 4 (j & 1) of x.
      if constexpr (kSplit > 1) {
        float* buf = sums + parity * Cfg::kSumFloats;
        parity ^= 1;
        if (part > 0) {
          float* dst = buf + ((part - 1) * Cfg::kRows + mrow) * kPass;
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[(n * 4 + j) * 32 + lane] = total[n][j];
        }
        // One barrier per tile: the buffer of the tile before last is read by part
        // 0 before it arrives here for the last one.
        consumer_barrier();
        if (part > 0) continue;
#pragma unroll
        for (int q = 1; q < kSplit; ++q) {
          const float* src = buf + ((q - 1) * Cfg::kRows + mrow) * kPass;
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) total[n][j] += src[(n * 4 + j) * 32 + lane];
        }
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = t.m0 + mrow + g + (j >> 1) * 8;
          const int r = n * 8 + c4 + (j & 1) * 4;
          if (m < p.M && r < t.rows)
            p.out[static_cast<size_t>(t.row0 + r) * p.M + m] =
                static_cast<uint16_t>(pack_bf16x2(total[n][j], 0.f) & 0xffffu);
        }
    }
    // Rows that no expert owns.
    const int mvec = p.M / 8;
    uint4* o4 = reinterpret_cast<uint4*>(p.out);
    for (int r = s_first[p.E] + blockIdx.x; r < p.N; r += gridDim.x)
      for (int c = threadIdx.x; c < mvec; c += kConsumers * 32)
        o4[static_cast<size_t>(r) * mvec + c] = make_uint4(0, 0, 0, 0);
  }
}

typedef void (*Kernel)(const CUtensorMap, const CUtensorMap, const Params);

struct Variant {
  Kernel kernel;
  size_t smem;
  int rows;
};

template <int kGroup, int kSplit, int kTiles>
Variant variant() {
  return Variant{matvec4_kernel<kGroup, kSplit, kTiles>, Config<kSplit, kTiles>::kSmem,
                 Config<kSplit, kTiles>::kRows};
}

template <int kGroup>
Variant pick(int split, int tiles) {
  if (split > 1) return tiles == 1 ? variant<kGroup, 4, 1>() : variant<kGroup, 2, 2>();
  return tiles == 1 ? variant<kGroup, 1, 1>()
                    : tiles == 2 ? variant<kGroup, 1, 2>() : variant<kGroup, 1, 4>();
}

Variant pick(int group, int split, int tiles) {
  return group == 32 ? pick<32>(split, tiles)
                     : group == 64 ? pick<64>(split, tiles) : pick<128>(split, tiles);
}

}  // namespace

cudaError_t setup_matvec4(const DeviceInfo&) {
  for (int group : {32, 64, 128})
    for (int split : {1, 2})
      for (int tiles : {1, 2, 4}) {
        const Variant v = pick(group, split, tiles);
        const cudaError_t e = cudaFuncSetAttribute(
            v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(v.smem));
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_matvec4(const Matvec4Args& a, const DeviceInfo& dev, cudaStream_t stream) {
  // Rows per pass: all of them with one matrix, else by the mean rows per expert
  // (an expert with more takes several passes, which re-read its weights from L2).
  const int matrices = std::min(a.E, a.N);
  const int64_t mean8 = a.E == 1 ? a.N : 4 * (static_cast<int64_t>(a.N) / matrices);
  int tiles = mean8 <= 8 ? 1 : mean8 <= 16 ? 2 : 4;
  const int64_t large = static_cast<int64_t>(matrices) * ((a.M + 127) / 128);
  const int split = tiles <= 2 && large < 4 * dev.num_sms ? 2 : 1;
  const Variant v = pick(a.G, split, tiles);
  CUtensorMap w_map, x_map;
  if (!make_map_u8_sw128(&w_map, a.packed, static_cast<uint64_t>(a.E) * a.M, a.C / 2, v.rows) ||
      !make_map_bf16_sw128(&x_map, a.x, a.N, a.C, 8))
    return cudaErrorInvalidValue;
  const int64_t most = (static_cast<int64_t>(matrices) + a.N / 8 + 1) *
                       ((a.M + v.rows - 1) / v.rows);
  const int grid = static_cast<int>(std::min<int64_t>(2 * dev.num_sms, most));
  const Params p{a.scales, a.offsets, a.out, a.N, a.E, a.M, a.C, dev.err_word};
  return launch_dependent(v.kernel, dim3(grid), dim3(kThreads), v.smem, stream, w_map, x_map, p);
}

}  // namespace lt
