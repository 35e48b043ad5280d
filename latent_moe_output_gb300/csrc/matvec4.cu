// latent_tail_expert_matvec4: products of expert-sorted rows with 4-bit weights
// that carry one scale per group of G columns.
//
//   out[r,m] = sum_c x[r,c] * (q[e,m,c] - 8) * s[e,m,c/G]
//            = sum_groups s[e,m,g] * ( sum_{c in g} x[r,c] * (q[e,m,c] - 8) )
//
// With the few rows per expert of a decode step the weights are read once and
// used at most a few times, so their stream bounds the call, and near it the
// instructions that unpack them: at the measured copy rate an SM receives 41 weights
// per clock at G = 32, has 128 instruction lanes per clock, and spends about two
// instructions per weight (64 % of the lanes).
// A 4-bit value masked out at bit 0 or 4 of a bf16 pattern is that integer times
// 2^-133 (subnormals and the first binade are one linear range), so one masking and
// one exact bf16 fused multiply-add per two weights give (q - 8) / 64: five logic
// operations for eight weights. The inner sums run on the tensor cores with these
// exact operands and FP32 accumulators: 16 weight rows x 16 columns against 8 rows
// of x per instruction. These warp-level instructions take their operands from
// registers, where the unpacked weights are; the tcgen05 ones would need them
// written back to shared memory first, and at 8 or 16 rows the tensor rate does not
// matter. Scales multiply the FP32 group sums; the factor 64 is applied at the end.
//
// Layout of the work. A tile is kRows = 32 to 256 weight rows of one expert,
// against up to 8 * kTiles rows of x (a pass). The CTAs walk over the tiles of
// the experts that have rows (found from the offsets at the start of the kernel).
// One warp streams weights and x through a ring of stages with TMA: a stage holds
// kSplit boxes of 256 columns (kRows x 128 bytes of weights, swizzled so that the
// eight rows of a fragment lie in different banks, 8 * kTiles rows of x, the scales). The
// eight other warps each own 32 weight rows (a fragment of x serves two of weights) and,
// with one box per stage, all of its columns: no warp then waits for another one.
// With several boxes a warp takes half of one, and the column parts are added in
// order through shared memory at the end of a tile: that makes enough tiles to fill
// the GPU from one matrix.
//
// Measured (GB300, launched back to back, weights of three calls in turn): 16 tokens
// with 8 of 256 experts of 2048 x 2048, G = 32 (about 103 experts read, 240 MB):
// 50 us = 4.8 TB/s, 71 % of the measured copy rate; 64 tokens: 94 us, 5.6 TB/s. The
// stream alone, without the arithmetic, takes 40 and 81 us; per stage a warp issues for
// 2500 cycles, waits for 700 and spends 250 between tiles. Which of them is the limit is
// not known: 60 % of the issue slots are used, 26 % of the tensor pipe, 71 % of the copy
// rate. One token with one matrix of 7168 x 2048, G = 128: 5.5 us, of which the weights'
// bytes are 1.1: the weights are first asked for after the wait for the kernel before and
// the experts' table, and a tile has two stages.
#include "block_launch.h"
#include "rows.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kConsumers = 8;  // warps
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kBoxCols = 256;  // columns per box: 128 bytes of weights
constexpr int kMaxStages = 8;
constexpr int kM = 2;  // fragments of 16 weight rows per warp
constexpr int kSmemPerSm = 204 * 1024;  // dynamic, without the experts' table
constexpr int table_bytes(int E) { return (E + 1) * 2 * static_cast<int>(sizeof(int)); }

template <int kSplit, int kTiles>
struct Config {
  // With one box per stage a warp takes all of its columns, else half of one box's.
  static constexpr int kHalves = kSplit == 1 ? 1 : 2;
  static constexpr int kParts = kSplit * kHalves;  // column parts of a stage
  static constexpr int kRowWarps = kConsumers / kParts;
  static constexpr int kRows = kRowWarps * 16 * kM;
  static constexpr int kCtasPerSm = 2;  // 96 registers
  static constexpr int kWeightBytes = kSplit * kRows * 128;
  static constexpr int kXBoxBytes = 8 * 128;  // 8 rows x 64 columns
  static constexpr int kXBytes = kSplit * kTiles * 4 * kXBoxBytes;
  // With one or two boxes per stage, 16 scales per row (32 bytes, a whole memory
  // sector) come with the first stage that needs them and serve group / 16 boxes; the
  // buffer belongs to a stage's slot, so it is free again no later than the slot is.
  // Otherwise eight scales per row and box, every time.
  static constexpr bool kPieces = kSplit <= 2;
  static constexpr int kPieceBytes = kPieces ? 32 : 16;
  static constexpr int kScaleBytes = (kPieces ? 1 : kSplit) * kRows * kPieceBytes;
  static constexpr int kStageBytes = kWeightBytes + kXBytes + kScaleBytes;
  // Column parts 1.. of a tile's sums.
  static constexpr int kSumBytes = (kParts - 1) * kRows * 8 * kTiles * 4;
  static constexpr int kFit = (kSmemPerSm / kCtasPerSm - kSumBytes - 1024) / kStageBytes;
  static constexpr int kStages = kFit > kMaxStages ? kMaxStages : kFit;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + kSumBytes + 1024;
  static_assert(kStages >= 2, "a ring needs two stages");
};

struct Params {
  const uint16_t* scales;
  const int32_t* offsets;
  uint16_t* out;
  int N, E, M, C;
  bool staged_scales;  // the scales come through the ring (their rows are whole 16-byte pieces)
  bool x_chunks;       // x has whole 64-column chunks: one copy brings a box's four
  uint32_t* err;
  RingLimits ring;
};

// Two of the eight values of a word, in the low four bits of each half (kHigh
// false) or the four bits above them: (q - 8) / 64 as two bf16 numbers, exact.
template <bool kHigh>
__device__ __forceinline__ uint32_t weight_pair(uint32_t w) {
  const uint32_t bits = w & (kHigh ? 0x00F000F0u : 0x000F000Fu);  // q * 2^-133 (* 16)
  uint32_t v;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;"
      : "=r"(v)
      : "r"(bits), "r"(kHigh ? 0x7D007D00u : 0x7F007F00u),  // 2^123, 2^127
        "r"(0xBE00BE00u));                                  // -8 / 64
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

// Barrier of the consumer warps; whether `ok` held for all of their threads.
__device__ __forceinline__ bool consumer_barrier(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "n"(kConsumers * 32)
      : "memory");
  return all != 0;
}

// Rows [row0, row0 + rows) of expert e against weight rows from m0 on.
struct __align__(16) Tile {
  int e, row0, rows, m0;
};

__device__ __forceinline__ Tile tile_at(int64_t tile, int mblocks, int rows_per_tile,
                                        int rows_per_pass, const int* s_first,
                                        const int* s_unit, int E) {
  // (a 64-bit division costs as much as the rest of this function)
  const int unit = tile >> 32 == 0 ? static_cast<uint32_t>(tile) / static_cast<uint32_t>(mblocks)
                                   : static_cast<int>(tile / mblocks);
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
  t.m0 = static_cast<int>(tile - static_cast<int64_t>(unit) * mblocks) * rows_per_tile;
  return t;
}

template <int kGroup, int kSplit, int kTiles>
__global__ void __launch_bounds__(kThreads, Config<kSplit, kTiles>::kCtasPerSm)
    matvec4_kernel(const __grid_constant__ CUtensorMap w_map,
                   const __grid_constant__ CUtensorMap x_map,
                   const __grid_constant__ CUtensorMap s_map, const Params p) {
  using Cfg = Config<kSplit, kTiles>;
  constexpr int kPass = 8 * kTiles;
  constexpr int kScales = kBoxCols / kGroup;  // per row and box
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[Cfg::kStages], empty_bar[Cfg::kStages];
  // The tile that begins with a stage, for the consumers: written before the stage's
  // barrier is armed, read after its wait, rewritten no earlier than the stage's slot.
  __shared__ Tile s_tile[Cfg::kStages];
  __shared__ int abort_flag;
  volatile int* abort_v = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // (shared memory is read through pointers, not asm, so that the compiler may move
  // the loads of one run of columns above the products of the last)
  uint8_t* ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
  float* sums = reinterpret_cast<float*>(ring_ptr + Cfg::kStages * Cfg::kStageBytes);
  int* s_first = reinterpret_cast<int*>(sums) + Cfg::kSumBytes / 4;  // first row of each expert
  int* s_unit = s_first + p.E + 1;                                   // passes before each expert

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

  constexpr int kStagesPerPiece = kGroup / 16 / kSplit > 1 ? kGroup / 16 / kSplit : 1;
  constexpr int kScalesAt = Cfg::kWeightBytes + Cfg::kXBytes;  // in a stage
  const int mblocks = (p.M + Cfg::kRows - 1) / Cfg::kRows;
  const int64_t tiles = static_cast<int64_t>(s_unit[p.E]) * mblocks;
  const int boxes = (p.C + kBoxCols - 1) / kBoxCols;
  const int steps = (boxes + kSplit - 1) / kSplit;  // stages per tile

  if (warp == kConsumers) {
    if (lane == 0) {
      uint32_t it = 0;  // stages issued
      uint32_t pieces = 0;  // scale pieces issued (one box per stage)
      bool ok = true;
      const int64_t copied = min(tiles, p.ring.copied);
      for (int64_t tile = blockIdx.x; ok && tile < copied; tile += gridDim.x) {
        const Tile t = tile_at(tile, mblocks, Cfg::kRows, kPass, s_first, s_unit, p.E);
        const int n_tiles = (t.rows + 7) / 8;
        for (int i = 0; i < steps; ++i, ++it) {
          const uint32_t s = it % Cfg::kStages;
          ok = mbar_wait(smem_u32(&empty_bar[s]), ((it / Cfg::kStages) & 1u) ^ 1u, p.err, abort_v,
                         p.ring.limit_ns);
          if (!ok) break;
          if (i == 0) s_tile[s] = t;
          const int live = min(kSplit, boxes - i * kSplit);
          const uint32_t bar = smem_u32(&full_bar[s]);
          const uint32_t st = ring + s * Cfg::kStageBytes;
          const bool piece = p.staged_scales && (!Cfg::kPieces || i % kStagesPerPiece == 0);
          mbar_arrive_expect_tx(
              bar, static_cast<uint32_t>(live) *
                           (Cfg::kRows * 128 + n_tiles * 4 * Cfg::kXBoxBytes) +
                       (piece ? (Cfg::kPieces ? 1 : live) * Cfg::kRows * Cfg::kPieceBytes : 0));
          if (Cfg::kPieces && piece) {
            tma_load_2d(ring + pieces % Cfg::kStages * Cfg::kStageBytes + kScalesAt, &s_map, bar,
                        i / kStagesPerPiece * 32, t.e * p.M + t.m0);
            ++pieces;
          }
          for (int j = 0; j < live; ++j) {
            const int c0 = (i * kSplit + j) * kBoxCols;
            tma_load_2d(st + j * Cfg::kRows * 128, &w_map, bar, c0 / 2, t.e * p.M + t.m0);
            if (!Cfg::kPieces && piece)  // from the piece that holds the box's first scale
              tma_load_2d(st + Cfg::kWeightBytes + Cfg::kXBytes + j * Cfg::kRows * 16, &s_map, bar,
                          (c0 / kGroup & ~7) * 2, t.e * p.M + t.m0);
            const uint32_t xs = st + Cfg::kWeightBytes + j * kTiles * 4 * Cfg::kXBoxBytes;
            for (int n = 0; n < n_tiles; ++n) {
              const uint32_t dst = xs + n * 4 * Cfg::kXBoxBytes;
              if (p.x_chunks) {
                tma_load_3d(dst, &x_map, bar, 0, t.row0 + n * 8, c0 / 64);
              } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  tma_load_2d(dst + c * Cfg::kXBoxBytes, &x_map, bar, c0 + c * 64, t.row0 + n * 8);
              }
            }
          }
        }
      }
      // The copies in flight land before the warp leaves; the consumers wait for them too,
      // but not after a wait that ran out.
      for (uint32_t i = it > Cfg::kStages ? it - Cfg::kStages : 0; i < it; ++i) {
        const uint32_t bar = smem_u32(&full_bar[i % Cfg::kStages]), parity = i / Cfg::kStages & 1u;
        if (mbar_try_wait(bar, parity)) continue;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else {
    constexpr int kRowWarps = Cfg::kRowWarps;
    constexpr int kRuns = 8 / Cfg::kHalves;         // runs of 32 columns per box and warp
    constexpr int kHalf = kScales / Cfg::kHalves;   // scales per row, box and warp
    constexpr int kWords = (kHalf + 1) / 2;
    const int part = warp / kRowWarps;              // column part of every stage
    const int box_in = part / Cfg::kHalves, half = part % Cfg::kHalves;  // its box and half
    const int mrow = warp % kRowWarps * 16 * kM;    // first weight row in the tile
    const int g = lane >> 2, c4 = lane & 3;
    // Column n of a fragment holds row (n >> 1) + 4 (n & 1) of the eight: lanes of
    // one quarter of the warp then read different halves of the swizzled rows.
    const int xrow = (g >> 1) + (g & 1) * 4;
    const int pitch = p.C / kGroup;  // scales per row
    uint32_t it = 0, pieces = 0;
    // Whether all stages have come. A lane whose wait runs out waits no more and releases
    // no stage, but takes part in the products, which are operations of whole warps; what
    // they make of a stage that did not come is not stored.
    bool ok = true;
    auto wait_full = [&](uint32_t s) {
      return mbar_wait(smem_u32(&full_bar[s]), (it / Cfg::kStages) & 1u, p.err, abort_v,
                       p.ring.limit_ns);
    };
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      ok = __all_sync(0xffffffffu, ok && wait_full(it % Cfg::kStages));
      Tile t{};  // (without rows: nothing is stored)
      if (ok) t = s_tile[it % Cfg::kStages];
      const int n_tiles = kTiles == 1 ? 1 : (t.rows + 7) / 8;
      float total[kM][kTiles][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[m][n][j] = 0.f;

      for (int i = 0; i < steps; ++i, ++it) {
        const uint32_t s = it % Cfg::kStages;
        if (ok && i > 0) ok = wait_full(s);
        const int box = i * kSplit + box_in;
        const int runs = min(kRuns, (p.C - box * kBoxCols) / 32 - half * kRuns);
        const uint8_t* st = ring_ptr + s * Cfg::kStageBytes;
        const uint8_t* wa = st + box_in * Cfg::kRows * 128 + (mrow + g) * 128 + c4 * 4;
        const uint8_t* xa =
            st + Cfg::kWeightBytes + box_in * kTiles * 4 * Cfg::kXBoxBytes + xrow * 128;
        // This warp's scales of the box: kHalf per row, two per register.
        uint32_t sc[2 * kM][kWords] = {};
        if (p.staged_scales) {
          if (Cfg::kPieces && i % kStagesPerPiece == 0) ++pieces;
          const uint32_t slot = Cfg::kPieces ? (pieces - 1) % Cfg::kStages : s;
          constexpr int kMask = Cfg::kPieceBytes / 2 - 1;  // scales in a piece
          const uint8_t* sa = ring_ptr + slot * Cfg::kStageBytes + kScalesAt +
                              ((Cfg::kPieces ? 0 : box_in * Cfg::kRows) + mrow + g) *
                                  Cfg::kPieceBytes +
                              ((box * kScales & kMask) + half * kHalf) * 2;
#pragma unroll
          for (int h = 0; h < 2 * kM; ++h) {
            if constexpr (kHalf == 8) {
              const uint4 v = *reinterpret_cast<const uint4*>(
                  sa + ((h >> 1) * 16 + (h & 1) * 8) * Cfg::kPieceBytes);
              sc[h][0] = v.x;
              sc[h][1] = v.y;
              sc[h][2] = v.z;
              sc[h][3] = v.w;
            } else if constexpr (kHalf == 4) {
              const uint2 v = *reinterpret_cast<const uint2*>(sa + h * 8 * Cfg::kPieceBytes);
              sc[h][0] = v.x;
              sc[h][1] = v.y;
            } else {
              sc[h][0] = kHalf == 2
                             ? *reinterpret_cast<const uint32_t*>(sa + h * 8 * Cfg::kPieceBytes)
                             : *reinterpret_cast<const uint16_t*>(sa + h * 8 * Cfg::kPieceBytes);
            }
          }
        } else if (runs > 0) {
          const int first = box * kScales + half * kHalf;
          const uint16_t* stile = p.scales + (static_cast<size_t>(t.e) * p.M + t.m0) * pitch;
#pragma unroll
          for (int h = 0; h < 2 * kM; ++h)
#pragma unroll
            for (int q = 0; q < kHalf; ++q)
              if (first + q < pitch) {  // (rows past the matrix are read from its last row)
                const int row = min(p.M - 1 - t.m0, mrow + g + h * 8);
                sc[h][q >> 1] |= static_cast<uint32_t>(__ldg(stile + row * pitch + first + q))
                                 << (16 * (q & 1));
              }
        }
        float acc[kM][kTiles][4];
        auto run = [&](int j) {  // j: run in the half box, known at compile time
          constexpr int kRunsPerGroup = kGroup / 32;
          const bool opens = j % kRunsPerGroup == 0, closes = (j + 1) % kRunsPerGroup == 0;
          const int chunk = half * kRuns + j;
          uint32_t lo[kM][4], hi[kM][4];  // fragments: values 0, 1, 4, 5 and 2, 3, 6, 7
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const uint8_t* at = wa + m * 16 * 128 + ((chunk ^ g) << 4);
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(at);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(at + 8 * 128);
            lo[m][0] = weight_pair<false>(w0);
            lo[m][1] = weight_pair<false>(w1);
            lo[m][2] = weight_pair<true>(w0);
            lo[m][3] = weight_pair<true>(w1);
            hi[m][0] = weight_pair<false>(w0 >> 8);
            hi[m][1] = weight_pair<false>(w1 >> 8);
            hi[m][2] = weight_pair<true>(w0 >> 8);
            hi[m][3] = weight_pair<true>(w1 >> 8);
          }
          const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            if (kTiles > 1 && n >= n_tiles) break;
            const uint4 v = *reinterpret_cast<const uint4*>(
                xa + (n * 4 + (chunk >> 1)) * Cfg::kXBoxBytes +
                ((((chunk & 1) * 4 + c4) ^ xrow) << 4));
            const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
            const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              if (opens)
                mma_bf16(acc[m][n], lo[m], b0, b1, zero);
              else
                mma_bf16(acc[m][n], lo[m], b0, b1, acc[m][n]);
              mma_bf16(acc[m][n], hi[m], b2, b3, acc[m][n]);
              if (closes) {
                const int q = j / kRunsPerGroup;
                const uint32_t u0 = sc[2 * m][q >> 1], u1 = sc[2 * m + 1][q >> 1];
                const float s0 = (q & 1) ? bf16_hi(u0) : bf16_lo(u0);
                const float s1 = (q & 1) ? bf16_hi(u1) : bf16_lo(u1);
                total[m][n][0] = fmaf(s0, acc[m][n][0], total[m][n][0]);
                total[m][n][1] = fmaf(s0, acc[m][n][1], total[m][n][1]);
                total[m][n][2] = fmaf(s1, acc[m][n][2], total[m][n][2]);
                total[m][n][3] = fmaf(s1, acc[m][n][3], total[m][n][3]);
              }
            }
          }
        };
        if (runs == kRuns) {
#pragma unroll
          for (int j = 0; j < kRuns; ++j) run(j);
        } else {  // (whole groups: C is a multiple of the group)
#pragma unroll
          for (int j = 0; j < kRuns - 1; ++j)
            if (j < runs) run(j);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_u32(&empty_bar[s]));
      }

      // Whether every stage has arrived for all warps whose sums a result has.
      if constexpr (Cfg::kParts == 1) ok = __all_sync(0xffffffffu, ok);
      if constexpr (Cfg::kParts > 1) {
        // The column parts of a row are added in order by part 0's warp.
        ok = consumer_barrier(ok);  // the last tile's sums have been read
        constexpr int kPerWarp = 16 * kM * 8 * kTiles;
        if (part > 0) {
          float* dst = sums + ((part - 1) * kRowWarps + warp % kRowWarps) * kPerWarp + lane;
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) dst[((m * kTiles + n) * 4 + j) * 32] = total[m][n][j];
        }
        consumer_barrier(true);
        if (part > 0) continue;
        for (int q = 0; q < Cfg::kParts - 1; ++q) {
          const float* src = sums + (q * kRowWarps + warp) * kPerWarp + lane;
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) total[m][n][j] += src[((m * kTiles + n) * 4 + j) * 32];
        }
      }
      if (!ok) continue;
      // Element (j, lane) of a fragment: weight row g + 8 (j >> 1), column
      // 2 c4 + (j & 1), i.e. row c4 + 4 (j & 1) of x.
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = t.m0 + mrow + m * 16 + g + (j >> 1) * 8;
            const int r = n * 8 + c4 + (j & 1) * 4;
            if (col < p.M && r < t.rows)
              p.out[static_cast<size_t>(t.row0 + r) * p.M + col] =
                  static_cast<uint16_t>(pack_bf16x2(64.f * total[m][n][j], 0.f) & 0xffffu);
          }
    }
    // Not before: CTAs of the next kernel would take the places of this one's that are
    // not resident yet (one matrix, one row: 6.3 against 5.7 us).
    pdl_launch_dependents();
    // Rows that no expert owns: before the first offset and from the last one on (all
    // rows where the offsets' running maximum leaves none).
    const int mvec = p.M / 8;
    uint4* o4 = reinterpret_cast<uint4*>(p.out);
    const int before = s_first[0], end = s_first[p.E];
    for (int i = blockIdx.x; i < before + p.N - end; i += gridDim.x) {
      const int r = i < before ? i : end + (i - before);
      for (int c = threadIdx.x; c < mvec; c += kConsumers * 32)
        o4[static_cast<size_t>(r) * mvec + c] = make_uint4(0, 0, 0, 0);
    }
  }
}

typedef void (*Kernel)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const Params);

struct Variant {
  Kernel kernel;
  size_t smem;
  int rows, ctas_per_sm, piece_bytes;
};

template <int kGroup, int kSplit, int kTiles>
Variant variant() {
  using Cfg = Config<kSplit, kTiles>;
  return Variant{matvec4_kernel<kGroup, kSplit, kTiles>, Cfg::kSmem, Cfg::kRows,
                 Cfg::kCtasPerSm, Cfg::kPieceBytes};
}

// split: 1 (whole boxes), 2 (two boxes per stage, 64 rows), 4 (the smallest tiles).
template <int kGroup>
Variant pick(int split, int tiles) {
  if (tiles == 1)
    return split == 1   ? variant<kGroup, 1, 1>()
           : split == 2 ? variant<kGroup, 2, 1>()
                        : variant<kGroup, 4, 1>();
  return split == 1 ? variant<kGroup, 1, 2>() : variant<kGroup, 2, 2>();
}

Variant pick(int group, int split, int tiles) {
  return group == 32 ? pick<32>(split, tiles)
                     : group == 64 ? pick<64>(split, tiles) : pick<128>(split, tiles);
}

}  // namespace

cudaError_t setup_matvec4(const DeviceInfo&) {
  for (int group : {32, 64, 128})
    for (int split : {1, 2, 4})
      for (int tiles : {1, 2}) {
        const Variant v = pick(group, split, tiles);
        const cudaError_t e = cudaFuncSetAttribute(
            v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
            static_cast<int>(v.smem) + table_bytes(kMaxExperts));
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_matvec4(const Matvec4Args& a, const DeviceInfo& dev, cudaStream_t stream) {
  // Tiles of 64 rows, of 32 where even those would leave a third of the SMs idle, as
  // long as tiles of 256 would not fill the GPU for a few rounds. (T tokens with 8 of
  // 256 experts of 2048 x 2048, us with tiles of 256 and of 64 rows: T = 3 20.3 and
  // 18.3, T = 6 28.5 and 28.6, T = 12 42.4 and 45.3. One row against one matrix, 64 and
  // 32 rows: 7168 x 2048 5.4 and 6.0, 2048 x 7168 11.8 and 9.5.)
  const int matrices = std::min(a.E, a.N);
  const int64_t tiles256 = static_cast<int64_t>(matrices) * ((a.M + 255) / 256);
  const int64_t tiles64 = static_cast<int64_t>(matrices) * ((a.M + 63) / 64);
  const bool narrow = 3 * tiles64 < 2 * dev.num_sms;
  const int split = tiles256 > 3 * dev.num_sms ? 1 : narrow ? 4 : 2;
  // Sixteen rows of x per pass instead of eight where an expert has more than twelve on
  // average: passes after the first read the weights from L2, and the second fragment
  // of x costs registers and a stage's space. (Mean rows 8: 42.5 us with eight and 46.2
  // with sixteen, 64 experts; mean 16: 66.4 and 61.6. One matrix, 24 rows: 9.6 and 8.3.)
  const int tiles = a.N / matrices > 12 && !narrow ? 2 : 1;
  const Variant v = pick(a.G, split, tiles);
  const uint64_t rows = static_cast<uint64_t>(a.E) * a.M;
  const uint64_t pitch = static_cast<uint64_t>(a.C / a.G) * 2;
  const bool staged = pitch % 16 == 0;
  const bool x_chunks = a.C % 64 == 0;
  CUtensorMap w_map, x_map, s_map;
  if (!make_map_u8(&w_map, a.packed, rows, a.C / 2, 128, v.rows) ||
      !(x_chunks ? make_map_bf16_rows64(&x_map, a.x, a.N, a.C, 8, 4)
                 : make_map_bf16_sw128(&x_map, a.x, a.N, a.C, 8)))
    return cudaErrorInvalidValue;
  if (!staged)
    s_map = w_map;  // not used
  else if (!make_map_u8(&s_map, a.scales, rows, pitch, v.piece_bytes, v.rows))
    return cudaErrorInvalidValue;
  const int64_t most = (static_cast<int64_t>(matrices) + a.N / 8 + 1) *
                       ((a.M + v.rows - 1) / v.rows);
  const int grid = static_cast<int>(std::min<int64_t>(v.ctas_per_sm * dev.num_sms, most));
  const Params p{a.scales, a.offsets, a.out, a.N, a.E, a.M, a.C, staged, x_chunks,
                 dev.err_word, a.ring};
  return launch_dependent(v.kernel, dim3(grid), dim3(kThreads),
                          v.smem + table_bytes(a.E), stream, w_map, x_map,
                          s_map, p);
}

}  // namespace lt
