// Products of expert-sorted rows with bf16 weights on the tensor cores, and their
// gradients (with r a row of expert e, W_e its weights):
//   kGated    h[r,f]   = a(sum_c x[r,c] W_e[f,c]) * sum_c x[r,c] W_e[F+f,c]
//   kRows     y[r,m]   = sum_k x[r,k] W_e[m,k]
//   kRowsT    dx[r,c]  = sum_m dy[r,m] W_e[m,c]
//   kWeights  dW_e[m,c] = sum_r dy[r,m] x[r,c]
//
// The row counts of experts are ragged, those of weights are not. So the weights are
// the MMA's M side, always 256 rows over a pair of CTAs (tcgen05 cta_group::2: each CTA
// loads its own 128 weight rows and half of the other operand), and the rows of an
// expert its N side, which an instruction takes in any multiple of 32 up to 256: an
// expert of n rows computes about n + 16 of them, where tiles of 256 (128) rows on the M
// side would compute n + 128 (n + 64) on average. An expert's rows are cut into the
// fewest tiles of at most 256, all of one size.
//
// kGated: the gate and the up row of a feature have to meet. A 5-D tensor map brings
// them into the tile in turns of eight (gate 0..7, up 0..7, gate 8..15, ...): rows of the
// accumulator are lanes of TMEM, so a lane finds the other projection of its feature
// eight lanes away, and one shuffle per two columns gives each lane both values of one
// (feature, row).
//
// kWeights: both operands run along M and N in memory (MN-major descriptors), and the
// sum runs over the rows. An expert whose count is not a multiple of 16 ends inside an
// MMA's 16 rows; what follows them are other experts' rows, of which one NaN would spoil
// the sum even against zeros. A warp of each CTA overwrites those rows of both operands
// with zeros in shared memory before the MMA reads them.
//
// Persistent, warp-specialized, one CTA per SM, 11 warps:
//   warp 0      producer: this CTA's operand boxes of a 128-deep block into a stage ring
//   warp 1      TMEM allocation; in the even CTA the MMA issuer (in both loops the whole warp
//               runs and one elected lane issues)
//   warps 2..9  epilogue; two accumulators, so the next tile's MMAs run meanwhile. The
//               lanes of TMEM are columns of the result: 32 rows at a time are turned
//               over in shared memory and leave in 16-byte pieces of whole row parts.
//               Two groups of four warps take every other 32 rows: one warp per scheduler
//               waits for its own shuffles and reciprocals most of the time
//   warp 10     kWeights: the zeros above; else zeros in the rows that no expert owns, with
//               the other warps' help once they are done
// Sums are FP32; results are rounded once.
#include "experts.cuh"

#include <algorithm>

namespace lt {
namespace {

enum Form { kGated, kRows, kRowsT, kWeights };

constexpr int kTileRows = 256;      // MMA N: rows of an expert (kWeights: columns)
// Depth of a stage: two pieces of 64, the span of a 128-byte swizzled row. Copies cost
// their issue, so a stage is deep and each operand comes in one copy of two pieces where its
// width is a multiple of 64 (8192 rows of 7168, 4096 columns: 347 us with stages of 64 and
// rows in boxes of 32, 307 with one box, 278 with stages of 128 in one copy per operand;
// since the producer's loop runs in a whole warp, two copies instead of one for all but the
// ragged end of other widths measure the same, and rows whose pitch is not a multiple of 128
// bytes cost by their extra requests: 8192 rows of 7176, F = 2040, 333 us against 285).
constexpr int kBlockK = 128;
constexpr uint32_t kPieceBytes = 128 * 128;  // 128 rows (or depths) of one piece
constexpr uint32_t kOperandBytes = 2 * kPieceBytes;
// (more than three, where tiles are small, measured the same; they hold the sums that pairs
// share)
constexpr int kMaxStages = 5;
constexpr int kGroups = 2;           // of four epilogue warps
constexpr int kSpareWarp = 2 + 4 * kGroups;
constexpr int kThreads = 32 * (kSpareWarp + 1);
constexpr uint32_t kTmemCols = 512;  // two accumulators
constexpr int kChunk = 32;           // rows turned over at a time

// Shared memory of one chunk. kRows: 32 rows of 128 bf16; the pad spreads them over banks.
constexpr int kPlainStride = 272;
// kGated: 32 rows of 64 products, and of 2 x 64 kept projections in bf16, or in 8 bits
// with 2 x 4 exponents. Strides of 8 (mod 32) words keep the two rows that a warp writes
// at once in different banks.
constexpr int kHiddenStride = 160;
constexpr int kKeptStride = 160;   // per projection
constexpr int kByteStride = 80;    // per projection
constexpr int kKeptAt = kChunk * kHiddenStride;
constexpr int kExponentsAt = kKeptAt + kChunk * 2 * kByteStride;

// kWeights: 16 rows of 64 bf16 for each warp.
constexpr int kSumStride = 144;

// Bytes for one group's chunk.
constexpr int turn_bytes(Form form, int saved_kind) {
  return form == kWeights ? 4 * 16 * kSumStride
         : form != kGated ? kChunk * kPlainStride
         : saved_kind == kSavedNone ? kKeptAt
         : saved_kind == kSavedBf16 ? kKeptAt + kChunk * 2 * kKeptStride
                                    : kExponentsAt + kChunk * 8;
}

struct Params {
  const int32_t* offsets;
  uint16_t* out;         // kGated: products [N,F]; kRows, kRowsT: [N,M]; kWeights: [E,M,C]
  void* saved;           // kGated: kept projections [N,2,F], bf16 or 8 bits, or null
  uint8_t* exponents;    // [N,2,groups]
  int N, E;
  int M;                 // kGated: F; kRows, kRowsT: columns of out; kWeights: its rows
  int K;                 // depth of a sum (kWeights: columns of out)
  int mblocks, cblocks;
  int tile_rows;         // most rows of a tile, at most kTileRows (kWeights: its columns)
  int parts;             // pairs of a cluster, which share a tile's sum
  int saved_kind;
  // Whether one copy brings both 64-column pieces of an operand: where its width is a
  // multiple of 64, so that a map may count the columns in pieces.
  bool whole_a, whole_b;
  int stages, stage_bytes, turn;
  uint32_t* err;
  RingLimits ring;
};

// Maps of operand B. kWeights: the first alone. Else boxes of 32, 64, 96 and 128 rows.
struct Maps {
  CUtensorMap map[4];
};

struct Tile {
  int e, row0, rows, m0, c0;
};

// The experts in the order of their tiles' cost, the largest first (see Walk).
struct Table {
  const int* first;  // [E+1] first row of each expert
  const int* order;  // experts
  const int* unit;   // passes over rows before each of `order` (not of kWeights)
};

// Rows of an expert's tiles: the fewest tiles of at most tile_rows rows, all of one size.
// (One tile as a rule, and no division: every CTA asks this of every expert.)
__device__ __forceinline__ int tiles_of(const Params& p, int n) {
  return n <= p.tile_rows ? (n > 0) : (n + p.tile_rows - 1) / p.tile_rows;
}
__device__ __forceinline__ int tile_size(int n, int tiles) {
  return ((tiles <= 1 ? n : (n + tiles - 1) / tiles) + 31) & ~31;
}

// Tile `tile` of the order: the features of one pass over an expert's rows, then the next
// pass. `at`, the place in the order, moves forward only.
template <Form kForm>
__device__ __forceinline__ Tile tile_at(const Params& p, int tile, int& at, const Table& s) {
  Tile t;
  if constexpr (kForm == kWeights) {
    const int per = p.mblocks * p.cblocks;
    at = tile / per;
    const int in = tile - at * per;
    t.e = s.order[at];
    t.row0 = s.first[t.e];
    t.rows = s.first[t.e + 1] - t.row0;
    t.m0 = in / p.cblocks * 256;
    t.c0 = in % p.cblocks * p.tile_rows;
  } else {
    const int unit = tile / p.mblocks;
    while (s.unit[at + 1] <= unit) ++at;
    t.e = s.order[at];
    const int n = s.first[t.e + 1] - s.first[t.e], i = unit - s.unit[at];
    const int tiles = (n + p.tile_rows - 1) / p.tile_rows;
    const int size = ((n + tiles - 1) / tiles + 31) & ~31;  // (tile_size without its branch)
    t.row0 = s.first[t.e] + i * size;
    t.rows = min(size, n - i * size);
    t.m0 = (tile - unit * p.mblocks) * (kForm == kGated ? 128 : 256);
    t.c0 = 0;
  }
  return t;
}

// The tiles of one cluster. Experts come in the order of their tiles' cost, and the
// clusters take turns forwards and backwards, so that what the first pays more in one turn
// it pays less in the next, and the last turn, which some clusters do not have, is of the
// cheapest tiles (1013 tokens, 6 of 60 experts, unevenly loaded, gated and kept in 8 bits:
// 81 us in the order of the experts, 74 like this).
struct Walk {
  int me, clusters, tiles, base = 0;
  bool back = false;
  __device__ Walk(int cluster, int n_clusters, int n_tiles)
      : me(cluster), clusters(n_clusters), tiles(n_tiles) {}
  __device__ __forceinline__ int tile() const { return base + (back ? clusters - 1 - me : me); }
  __device__ __forceinline__ bool more() const { return tile() < tiles; }
  __device__ __forceinline__ void next() {
    base += clusters;
    back = !back;
  }
};

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// What a producer has issued (words, in shared memory).
struct Issued {
  uint32_t blocks;
  uint32_t bytes[kMaxStages];  // of the last block in a stage, on full_bar (0: on tail_bar)
  uint32_t tails[kMaxStages];  // blocks in a stage on tail_bar
};

// Waits, in the even CTA, for the copies of both CTAs of a pair. The two may have issued
// different numbers of blocks when a wait ran out, and a barrier completes only with as many
// bytes as the even CTA expected: what the odd CTA has issued beyond the even one is expected
// here, and what it has not issued is taken off. A CTA issues a block only after the MMAs of
// the one before it in the stage, so no more than the last `stages` blocks are open.
__device__ __noinline__ void drain_copies(uint64_t* full_bar, int stages, const Issued& even,
                                          const Issued& odd) {
  const int own = static_cast<int>(even.blocks), other = static_cast<int>(odd.blocks);
  const int most = max(own, other);
  for (int it = max(0, most - stages); it < most; ++it) {
    const int s = it % stages;
    const uint32_t bar = smem_u32(&full_bar[s]);
    if (it >= own) {
      if (odd.bytes[s] == 0) continue;
      mbar_arrive_expect_tx(bar, odd.bytes[s]);
    } else if (it >= other && even.bytes[s] != 0) {
      mbar_complete_tx(bar, even.bytes[s]);
    }
    wait_drain(bar, static_cast<uint32_t>(it / stages) & 1u);
  }
}

// mbar_wait for the copy of a block that the producer may come to much later: the limit
// begins again whenever `blocks`, what it has issued, has grown.
__device__ __forceinline__ bool wait_behind(uint32_t bar, uint32_t parity, uint32_t* err,
                                            volatile int* abort_flag, uint64_t limit_ns,
                                            const volatile uint32_t* blocks) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = global_timer_ns();
  uint32_t seen = *blocks;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    const uint32_t now = *blocks;
    if (now != seen) {
      seen = now;
      t0 = global_timer_ns();
    } else if (global_timer_ns() - t0 > limit_ns) {
      atomicOr(err, kErrWaitTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void group_barrier(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

template <Form kForm, int kAct>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const __grid_constant__ CUtensorMap a_map,
                  const __grid_constant__ Maps b_maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[kMaxStages];   // even CTA: both CTAs' stage landed
  __shared__ uint64_t empty_bar[kMaxStages];  // stage consumed by the pair's MMAs
  __shared__ uint64_t tail_bar[kMaxStages];   // kWeights: this CTA's last block landed
  __shared__ uint64_t fixed_bar[kMaxStages];  // even CTA: both CTAs' zeros are in place
  __shared__ uint64_t accf_bar[2];            // accumulator ready (both CTAs)
  __shared__ uint64_t acce_bar[2];            // even CTA: accumulator drained by both
  __shared__ uint64_t drain_bar;              // even CTA: MMAs before an abort are done
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int zero_next;    // rows without an expert that have been handed out
  __shared__ int part_failed;  // a pair's sum did not come (first pair of a cluster)
  // For the wind-down after a wait that ran out (see drain_copies): blocks that this CTA's
  // producer has issued, the bytes of the last one in each stage that count on the even CTA's
  // full_bar, and the blocks in each stage that counted on this CTA's tail_bar.
  __shared__ Issued issued, odd_issued;  // (odd_issued: in the even CTA, the odd one's)
  __shared__ int wind_down;              // a wait ran out in some CTA of the cluster
  volatile int* abort_v = &abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_rank());
  const int rank = cta & 1, even = cta & ~1, part = cta >> 1;
  const int cluster = static_cast<int>(blockIdx.x) / (2 * p.parts);
  const int n_clusters = static_cast<int>(gridDim.x) / (2 * p.parts);
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const int stages = p.stages;
  uint8_t* turn_ptr = smem_raw + (ring - raw) + static_cast<uint32_t>(stages * p.stage_bytes);
  int* s_first = reinterpret_cast<int*>(turn_ptr + kGroups * p.turn);
  int* s_unit = s_first + p.E + 1;
  int* s_order = s_unit + p.E + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
      mbar_init(smem_u32(&tail_bar[s]), 1);
      mbar_init(smem_u32(&fixed_bar[s]), 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&accf_bar[a]), 1);
      mbar_init(smem_u32(&acce_bar[a]), 2 * 4 * kGroups);  // one per epilogue warp of the pair
    }
    mbar_init(smem_u32(&drain_bar), 1);
    abort_flag = 0;
    issued = Issued{};
    wind_down = 0;
    part_failed = 0;
    zero_next = 0;
    mbar_fence_init();
    tma_prefetch_map(&a_map);
    tma_prefetch_map(&b_maps.map[0]);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), kTmemCols);
  pdl_wait();
  load_experts(p.offsets, p.N, p.E, s_first);
  const int live = order_experts(p.E, s_order, [&](int e) {
    const int n = s_first[e + 1] - s_first[e];
    if (kForm == kWeights)  // experts without rows get zeros
      return min(kClasses, max(1, (n + kBlockK - 1) / kBlockK));
    return n == 0 ? 0 : tile_size(n, tiles_of(p, n)) / 32;
  });
  if (kForm != kWeights)
    sum_units(live, s_unit, [&](int i) {
      return tiles_of(p, s_first[s_order[i] + 1] - s_first[s_order[i]]);
    });
  const Table table{s_first, s_order, s_unit};
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  int tiles = kForm == kWeights ? p.E * p.mblocks * p.cblocks : s_unit[live] * p.mblocks;
  // Pairs that share a sum meet once: such a launch has a cluster for every tile.
  if (p.parts > 1) tiles = min(tiles, n_clusters);
  // Blocks of a tile's sum, and whether the last one of kWeights needs zeros.
  auto blocks_of = [&](const Tile& t) {
    return ((kForm == kWeights ? t.rows : p.K) + kBlockK - 1) / kBlockK;
  };
  // This pair's part of them.
  auto first_block = [&](int nkb, int i) { return nkb * i / p.parts; };
  auto needs_zeros = [&](const Tile& t) { return kForm == kWeights && (t.rows & 15) != 0; };
  // Rows of an MMA's N side.
  auto width_of = [&](const Tile& t) {
    return kForm == kWeights ? p.tile_rows : (t.rows + 31) & ~31;
  };

  // Zeros in the rows that no expert owns: rows are handed out one by one, to the spare warp
  // from the start and to the others when they have nothing else to do (8000 tokens with 6 of
  // 60 experts, nine choices of ten without one, gated and kept in 8 bits: 133 us by the
  // spare warp alone, 115 like this).
  auto zero_rows = [&]() {
    const int before = s_first[0], none = before + p.N - s_first[p.E];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    while (true) {
      int64_t i = 0;
      if (lane == 0) i = blockIdx.x + static_cast<int64_t>(atomicAdd(&zero_next, 1)) * gridDim.x;
      i = __shfl_sync(0xffffffffu, i, 0);
      if (i >= none) break;
      const size_t r = static_cast<size_t>(i < before ? i : s_first[p.E] + (i - before));
      uint4* o = reinterpret_cast<uint4*>(p.out + r * p.M);
      for (int c = lane; c < p.M / 8; c += 32) o[c] = zero;
      if (kForm == kGated && p.saved_kind == kSavedBf16) {
        uint4* k = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.saved) + r * 2 * p.M);
        for (int c = lane; c < p.M / 4; c += 32) k[c] = zero;
      } else if (kForm == kGated && p.saved_kind == kSaved8) {
        uint4* k = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.saved) + r * 2 * p.M);
        for (int c = lane; c < p.M / 8; c += 32) k[c] = zero;
        const int groups = 2 * ((p.M + kGroup8 - 1) / kGroup8);
        for (int c = lane; c < groups; c += 32) p.exponents[r * groups + c] = 0;
      }
    }
  };

  bool joined = false;  // whether this warp has met the others of the cluster for the sums
  if (warp == 0) {
    {
      // ---------------- producer (this CTA's halves; the whole warp, one lane issues) ------
      int at = 0, s = 0;
      uint32_t round = 0;
      int blocks = 0;
      const int copied = static_cast<int>(min(static_cast<int64_t>(tiles), p.ring.copied));
      bool alive = true;
      for (Walk walk(cluster, n_clusters, copied); alive && walk.more(); walk.next()) {
        const Tile t = tile_at<kForm>(p, walk.tile(), at, table);
        const int nkb = blocks_of(t);
        const int half = width_of(t) / 2;
        const int box = (half + 31) / 32;  // in 32 rows
        const CUtensorMap* b_map = &b_maps.map[kForm == kWeights ? 0 : box - 1];
        const uint32_t b_piece = kForm == kWeights ? kPieceBytes : box * 4096u;
        const uint32_t bytes = kOperandBytes + 2 * b_piece;
        for (int kb = first_block(nkb, part); kb < first_block(nkb, part + 1); ++kb) {
          alive = __all_sync(0xffffffffu,
                             mbar_wait_cluster(smem_u32(&empty_bar[s]), (round & 1u) ^ 1u, p.err,
                                               abort_v, p.ring.limit_ns));
          if (!alive) break;
          const uint32_t a = ring + static_cast<uint32_t>(s * p.stage_bytes), b = a + kOperandBytes;
          const int k0 = kb * kBlockK;
          const bool tail = kForm == kWeights && kb == nkb - 1 && needs_zeros(t);
          const bool issue = elect_one();
          ++blocks;
          if (issue) {
            issued.blocks = blocks;
            issued.bytes[s] = tail ? 0 : bytes;
            if (tail) ++issued.tails[s];
          }
          if (issue && tail) {
            // Completes on this CTA's own barrier, for the warp that puts the zeros in.
            const uint32_t bar = smem_u32(&tail_bar[s]);
            if (rank == 0) mbar_arrive(smem_u32(&full_bar[s]));
            mbar_arrive_expect_tx(bar, 2 * kOperandBytes);
            const int m = t.m0 + rank * 128, c = t.c0 + rank * half, r = t.row0 + k0;
            if (p.whole_a) {
              tma_load_3d(a, &a_map, bar, 0, r, m / 64);
            } else {
              tma_load_2d(a, &a_map, bar, m, r);
              tma_load_2d(a + kPieceBytes, &a_map, bar, m + 64, r);
            }
            if (p.whole_b) {
              tma_load_3d(b, b_map, bar, 0, r, c / 64);
            } else {
              tma_load_2d(b, b_map, bar, c, r);
              tma_load_2d(b + kPieceBytes, b_map, bar, c + 64, r);
            }
          } else if (issue) {
            const uint32_t bar = map_to_rank(smem_u32(&full_bar[s]), even);
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), 2 * bytes);
            const int m = t.m0 + rank * (kForm == kGated ? 64 : 128);
            if constexpr (kForm == kGated) {
              const int eight = t.e * (p.M / 4) + m / 8;  // eights of rows, all experts'
              if (p.whole_a) {
                tma_load_5d_pair(a, &a_map, bar, 0, 0, 0, eight, k0 / 64);
              } else {
                tma_load_4d_pair(a, &a_map, bar, k0, 0, 0, eight);
                tma_load_4d_pair(a + kPieceBytes, &a_map, bar, k0 + 64, 0, 0, eight);
              }
            } else if constexpr (kForm == kRows) {
              if (p.whole_a) {
                tma_load_4d_pair(a, &a_map, bar, 0, m, k0 / 64, t.e);
              } else {
                tma_load_3d_pair(a, &a_map, bar, k0, m, t.e);
                tma_load_3d_pair(a + kPieceBytes, &a_map, bar, k0 + 64, m, t.e);
              }
            } else if constexpr (kForm == kRowsT) {
              if (p.whole_a) {
                tma_load_4d_pair(a, &a_map, bar, 0, k0, m / 64, t.e);
              } else {
                tma_load_3d_pair(a, &a_map, bar, m, k0, t.e);
                tma_load_3d_pair(a + kPieceBytes, &a_map, bar, m + 64, k0, t.e);
              }
            } else {
              if (p.whole_a) {
                tma_load_3d_pair(a, &a_map, bar, 0, t.row0 + k0, m / 64);
              } else {
                tma_load_2d_pair(a, &a_map, bar, m, t.row0 + k0);
                tma_load_2d_pair(a + kPieceBytes, &a_map, bar, m + 64, t.row0 + k0);
              }
            }
            // (kWeights: columns c of the rows from r on; else rows r, columns from k0 on)
            const int c = t.c0 + rank * half, r = t.row0 + (kForm == kWeights ? k0 : rank * half);
            if (p.whole_b) {
              tma_load_3d_pair(b, b_map, bar, 0, r, (kForm == kWeights ? c : k0) / 64);
            } else {
              tma_load_2d_pair(b, b_map, bar, kForm == kWeights ? c : k0, r);
              tma_load_2d_pair(b + b_piece, b_map, bar, (kForm == kWeights ? c : k0) + 64, r);
            }
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            ++round;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------- pair MMA issuer (the whole warp, one lane issues) ----------------
      int at = 0, s = 0;
      uint32_t round = 0, fixed_phase = 0, use = 0;
      bool alive = true;
      // One thread issues all MMAs, and one of 256 x 256 x 16 takes 128 cycles: descriptors
      // are kept ready, so that an issue is two additions (with descriptors put together for
      // each, 160 cycles passed between two MMAs whatever their size).
      constexpr bool kMajorA = kForm == kGated || kForm == kRows, kMajorB = kForm != kWeights;
      const uint32_t a_base = kMajorA ? umma_desc_lo(ring) : umma_desc_lo(ring, kPieceBytes);
      const uint32_t b_base = kMajorB ? umma_desc_lo(ring + kOperandBytes)
                                      : umma_desc_lo(ring + kOperandBytes, kPieceBytes);
      const uint32_t stage_step = static_cast<uint32_t>(p.stage_bytes) >> 4;
      uint32_t a_lo = a_base, b_lo = b_base;
      auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu,
                          mbar_wait_cluster(bar, parity, p.err, abort_v, p.ring.limit_ns));
      };
      for (Walk walk(cluster, n_clusters, tiles); alive && walk.more(); walk.next()) {
        const Tile t = tile_at<kForm>(p, walk.tile(), at, table);
        const int nkb = blocks_of(t);
        if (nkb == 0) continue;
        const int acc = static_cast<int>(use & 1u);
        if (!wait_all(smem_u32(&acce_bar[acc]), ((use >> 1) & 1u) ^ 1u)) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * kTileRows);
        const uint32_t idesc = umma_idesc_bf16(256, width_of(t)) |
                               (kForm == kRowsT || kForm == kWeights ? kUmmaTransposeA : 0u) |
                               (kForm == kWeights ? kUmmaTransposeB : 0u);
        // Sixteenths of the bytes between the pieces of a K-major operand B, and of a step.
        const uint32_t b_piece = static_cast<uint32_t>((width_of(t) / 2 + 31) / 32) * 256u;
        auto a_step = [](int k) {
          return kMajorA ? 2u * (k & 3) + (kPieceBytes >> 4) * (k >> 2) : 128u * k;
        };
        auto b_step = [&](int k) { return kMajorB ? 2u * (k & 3) + b_piece * (k >> 2) : 128u * k; };
        const int kb0 = first_block(nkb, part), kb1 = first_block(nkb, part + 1);
        const int depth = kForm == kWeights ? t.rows : p.K;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_all(smem_u32(&full_bar[s]), round & 1u)) {
            alive = false;
            break;
          }
          const uint32_t first = kb != kb0 ? 1u : 0u;
          if (depth - kb * kBlockK >= kBlockK) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kBlockK / 16; ++k)
                umma_bf16_pair_lo(d, a_lo + a_step(k), b_lo + b_step(k), idesc,
                                  k == 0 ? first : 1u);
              umma_commit_pair(smem_u32(&empty_bar[s]), 0x3 << even);
            }
          } else {  // the last block
            if (needs_zeros(t)) {
              if (!wait_all(smem_u32(&fixed_bar[s]), fixed_phase >> s & 1u)) {
                alive = false;
                break;
              }
              fixed_phase ^= 1u << s;
            }
            tc_fence_after();
            const int steps = (depth - kb * kBlockK + 15) >> 4;
            if (elect_one()) {
#pragma unroll 1
              for (int k = 0; k < steps; ++k)
                umma_bf16_pair_lo(d, a_lo + a_step(k), b_lo + b_step(k), idesc,
                                  k == 0 ? first : 1u);
              umma_commit_pair(smem_u32(&empty_bar[s]), 0x3 << even);
            }
          }
          __syncwarp();
          a_lo += stage_step;
          b_lo += stage_step;
          if (++s == stages) {
            s = 0;
            ++round;
            a_lo = a_base;
            b_lo = b_base;
          }
        }
        if (!alive) break;  // (a sum that is not whole is not handed on)
        if (elect_one()) umma_commit_pair(smem_u32(&accf_bar[acc]), 0x3 << even);
        __syncwarp();
        ++use;
      }
    }
    __syncwarp();
  } else if (warp == kSpareWarp) {
    if constexpr (kForm == kWeights) {
      // ---------------- zeros behind an expert's last row ----------------
      int at = 0, it = 0;
      uint32_t phase = 0;
      bool alive = true;
      for (Walk walk(cluster, n_clusters, tiles); alive && walk.more(); walk.next()) {
        const Tile t = tile_at<kForm>(p, walk.tile(), at, table);
        const int nkb = blocks_of(t), end = first_block(nkb, part + 1);
        it += end - first_block(nkb, part);
        if (!needs_zeros(t) || end != nkb) continue;
        const int s = (it - 1) % stages;
        const int from = t.rows - (blocks_of(t) - 1) * kBlockK, to = (from + 15) & ~15;
        // The blocks before this one may take any time; the limit is of the one wait.
        alive = __all_sync(0xffffffffu,
                           wait_behind(smem_u32(&tail_bar[s]), phase >> s & 1u, p.err, abort_v,
                                       p.ring.limit_ns, &issued.blocks));
        if (!alive) break;
        phase ^= 1u << s;
        // Four boxes of 128 rows of 128 bytes (the swizzle stays within a row).
        uint8_t* st = smem_raw + (ring - raw) + static_cast<uint32_t>(s * p.stage_bytes);
        for (int i = lane; i < (to - from) * 32; i += 32) {
          const int row = from + (i >> 5), box = (i >> 3) & 3, piece = i & 7;
          *reinterpret_cast<uint4*>(st + box * kPieceBytes + row * 128 + piece * 16) =
              make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          const uint32_t bar = smem_u32(&fixed_bar[s]);
          mbar_arrive_remote(map_to_rank(bar, even));
        }
      }
    } else {
      zero_rows();
    }
  } else {
    // ---------------- epilogue (warps 2..9) ----------------
    const int q = warp & 3;  // the quarter of TMEM's lanes that this warp may access
    const int group = (warp - 2) >> 2;
    const int tid = (threadIdx.x - 64) & 127;  // in the group
    uint8_t* buf = turn_ptr + group * p.turn;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    auto release_acc = [&](int a) {  // accumulator read: back to the MMA issuer
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar = smem_u32(&acce_bar[a]);
        if (rank == 0)
          mbar_arrive(bar);
        else
          mbar_arrive_remote(map_to_rank(bar, even));
      }
    };
    // The other pairs' sums of 32 rows, in their order.
    auto add_parts = [&](const Tile& t, int ch, float (&v)[32]) {
      const int nt = width_of(t);
      const float* from = reinterpret_cast<const float*>(smem_raw + (ring - raw)) +
                          ch * kChunk * 128 + q * 32 + lane;
      for (int i = 1; i < p.parts; ++i, from += nt * 128)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += from[j * 128];
    };
    int at = 0;
    uint32_t use = 0;
    bool alive = true;
    for (Walk walk(cluster, n_clusters, tiles); alive && walk.more(); walk.next()) {
      const Tile t = tile_at<kForm>(p, walk.tile(), at, table);
      const bool any = blocks_of(t) != 0;
      const int acc = static_cast<int>(use & 1u);
      const uint32_t dcol = tmem + lane_base + static_cast<uint32_t>(acc * kTileRows);
      if (any) {
        // Every warp's waits end alike: the flag that one sets ends the others' too.
        alive = __all_sync(0xffffffffu,
                           mbar_wait_cluster(smem_u32(&accf_bar[acc]), (use >> 1) & 1u, p.err,
                                             abort_v, p.ring.limit_ns));
        if constexpr (kForm != kWeights) {
          uint32_t all;  // a group's warps turn rows over together
          asm volatile(
              "{\n\t.reg .pred p, q;\n\t"
              "setp.ne.u32 p, %1, 0;\n\t"
              "bar.red.and.pred q, %2, 128, p;\n\t"
              "selp.u32 %0, 1, 0, q;\n\t}"
              : "=r"(all)
              : "r"(static_cast<uint32_t>(alive)), "r"(1 + group)
              : "memory");
          alive = all != 0;
        }
        if (p.parts > 1) {
          // All pairs' products are done, so the first pair's stages are free: the others
          // put their sums there, [row][lane] for each pair and CTA.
          __syncwarp();
          cluster_sync();
          const int nt = width_of(t);
          if (part > 0 && alive) {
            tc_fence_after();
            const uint32_t to = map_to_rank(
                ring + (static_cast<uint32_t>(part - 1) * nt * 128 + q * 32 + lane) * 4, rank);
            for (int ch = group; ch * kChunk < nt; ch += kGroups) {
              float v[32];
              __syncwarp();
              tmem_ld32(dcol + static_cast<uint32_t>(ch * kChunk), v);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                st_dsmem_f32(to + static_cast<uint32_t>(ch * kChunk + j) * 512, v[j]);
            }
          } else if (part > 0 && lane == 0) {
            st_dsmem_u32(map_to_rank(smem_u32(&part_failed), rank), 1);
          }
          __syncwarp();
          cluster_sync();
          joined = true;
          if (part > 0 || *const_cast<volatile int*>(&part_failed) != 0) break;
        }
        if (!alive) break;
        tc_fence_after();
        ++use;
      }
      const int chunks = width_of(t) / kChunk;
      if constexpr (kForm == kWeights) {
        // Lanes are rows of dW_e, columns of TMEM its columns. 64 columns at a time go through
        // shared memory, half of the rows first, so that a store is of four rows' 128 bytes
        // and not of 32 rows' 16 (product of 60 experts of 91 rows, 1448 x 712, both gradients:
        // 102 us with pieces of 32 bytes, 96 with 64, 94 with 128).
        const int m0 = t.m0 + rank * 128 + q * 32;
        uint16_t* dst = p.out + (static_cast<size_t>(t.e) * p.M + m0) * p.K + t.c0;
        uint8_t* own = buf + q * 16 * kSumStride;
        if (any && 2 * group >= chunks) release_acc(acc);
        for (int ch = 2 * group; ch < chunks; ch += 2 * kGroups) {
          float v[2][32] = {};
          __syncwarp();
          if (any) {
            tmem_ld32(dcol + static_cast<uint32_t>(ch * kChunk), v[0]);
            if (ch + 1 < chunks) tmem_ld32(dcol + static_cast<uint32_t>((ch + 1) * kChunk), v[1]);
            if (ch + 2 * kGroups >= chunks) release_acc(acc);
            if (p.parts > 1) {
              add_parts(t, ch, v[0]);
              if (ch + 1 < chunks) add_parts(t, ch + 1, v[1]);
            }
          }
          const int c = (lane & 7) * 8;
          const bool in = ch * kChunk + c < p.tile_rows && t.c0 + ch * kChunk + c < p.K;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __syncwarp();  // the last rows have been read
            if (lane >> 4 == h) {
#pragma unroll
              for (int g = 0; g < 8; ++g)
                *reinterpret_cast<uint4*>(own + (lane & 15) * kSumStride + g * 16) =
                    pack8(*reinterpret_cast<const float(*)[8]>(&v[g >> 2][(g & 3) * 8]));
            }
            __syncwarp();
            if (in) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = i * 4 + (lane >> 3);
                if (m0 + h * 16 + r < p.M)
                  *reinterpret_cast<uint4*>(dst + static_cast<size_t>(h * 16 + r) * p.K +
                                            ch * kChunk + c) =
                      *reinterpret_cast<const uint4*>(own + r * kSumStride + c * 2);
              }
            }
          }
        }
      } else {
        if (group >= chunks) release_acc(acc);
        for (int ch = group; ch < chunks; ch += kGroups) {
          float v[32];
          __syncwarp();
          tmem_ld32(dcol + static_cast<uint32_t>(ch * kChunk), v);
          if (ch + kGroups >= chunks) release_acc(acc);
          if (p.parts > 1) add_parts(t, ch, v);
          group_barrier(group);  // the last chunk has been read
          const int live = min(kChunk, t.rows - ch * kChunk);  // rows of the chunk
          const size_t row = static_cast<size_t>(t.row0) + ch * kChunk;
          if constexpr (kForm != kGated) {
            uint8_t* at = buf + q * 64 + lane * 2;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              *reinterpret_cast<uint16_t*>(at + j * kPlainStride) =
                  static_cast<uint16_t>(pack_bf16x2(v[j], 0.f));
            group_barrier(group);
            const int m = t.m0 + rank * 128 + (tid & 15) * 8;
            if (m < p.M) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = (tid >> 4) + i * 8;
                if (r < live)
                  *reinterpret_cast<uint4*>(p.out + (row + r) * p.M + m) =
                      *reinterpret_cast<const uint4*>(buf + r * kPlainStride + (tid & 15) * 16);
              }
            }
          } else {
            // Lane: gate (half 0) or up (half 1) of feature `f` of this CTA's 64.
            const int half = (lane >> 3) & 1;
            const int f = q * 16 + ((lane >> 4) << 3) + (lane & 7);
            if (p.saved_kind == kSavedBf16) {
              uint8_t* at = buf + kKeptAt + half * kKeptStride + f * 2;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                *reinterpret_cast<uint16_t*>(at + j * 2 * kKeptStride) =
                    static_cast<uint16_t>(pack_bf16x2(v[j], 0.f));
            } else if (p.saved_kind == kSaved8) {
              // A group is the 16 lanes of one projection. Behind the last feature the tile
              // holds other rows' values; F is a multiple of 8, so half a group.
              const bool past = t.m0 + rank * 64 + f >= p.M;
              uint8_t* at = buf + kKeptAt + half * kByteStride + f;
              uint8_t* eat = buf + kExponentsAt + half * 4 + q;
              // The exponent goes by the upper 16 bits of the largest magnitude: two
              // columns' maxima in one word.
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                uint32_t top = past ? 0u
                                    : __byte_perm(__float_as_uint(v[j]), __float_as_uint(v[j + 1]),
                                                  0x7632) & 0x7FFF7FFFu;
                top = __vmaxs2(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = __vmaxs2(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = __vmaxs2(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = __vmaxs2(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const uint32_t e0 = exponent8(top & 0xFFFFu), e1 = exponent8(top >> 16);
                at[j * 2 * kByteStride] = integer8(v[j], e0);
                at[(j + 1) * 2 * kByteStride] = integer8(v[j + 1], e1);
                if ((lane & 23) == 0) {
                  eat[j * 8] = static_cast<uint8_t>(e0);
                  eat[j * 8 + 8] = static_cast<uint8_t>(e1);
                }
              }
            }
            uint8_t* at = buf + half * kHiddenStride + f * 2;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float other = __shfl_xor_sync(0xffffffffu, half ? v[2 * j] : v[2 * j + 1], 8);
              const float g = half ? other : v[2 * j], u = half ? v[2 * j + 1] : other;
              const float h = activation<kAct>(g) * u;
              *reinterpret_cast<uint16_t*>(at + 2 * j * kHiddenStride) =
                  static_cast<uint16_t>(pack_bf16x2(h, 0.f));
            }
            group_barrier(group);
            const int f0 = t.m0 + rank * 64;
            {
              const int c = (tid & 7) * 8;
              if (f0 + c < p.M) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int r = (tid >> 3) + i * 16;
                  if (r < live)
                    *reinterpret_cast<uint4*>(p.out + (row + r) * p.M + f0 + c) =
                        *reinterpret_cast<const uint4*>(buf + r * kHiddenStride + c * 2);
                }
              }
            }
            if (p.saved_kind == kSavedBf16) {
              const int c = (tid & 7) * 8, h = (tid >> 3) & 1;
              if (f0 + c < p.M) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int r = (tid >> 4) + i * 8;
                  if (r < live)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.saved) +
                                              ((row + r) * 2 + h) * p.M + f0 + c) =
                        *reinterpret_cast<const uint4*>(buf + kKeptAt +
                                                        (r * 2 + h) * kKeptStride + c * 2);
                }
              }
            } else if (p.saved_kind == kSaved8) {
              const int c = (tid & 7) * 8, h = (tid >> 3) & 1;
              if (f0 + c < p.M) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int r = (tid >> 4) + i * 8;
                  if (r < live)
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.saved) +
                                              ((row + r) * 2 + h) * p.M + f0 + c) =
                        *reinterpret_cast<const uint2*>(buf + kKeptAt +
                                                        (r * 2 + h) * kByteStride + c);
                }
              }
              const int groups = (p.M + kGroup8 - 1) / kGroup8;
              const int g0 = f0 / kGroup8 + (tid & 3);
              if (g0 < groups) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int at2 = (tid >> 2) + i * 32, r = at2 >> 1, h2 = at2 & 1;
                  if (r < live)
                    p.exponents[((row + r) * 2 + h2) * groups + g0] =
                        buf[kExponentsAt + r * 8 + h2 * 4 + (tid & 3)];
                }
              }
            }
          }
        }
      }
    }
  }

  if (p.parts > 1 && !joined) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  __syncwarp();
  if (kForm != kWeights) zero_rows();
  // Neither CTA may leave while the pair's MMAs could still read its shared memory or
  // write its TMEM, or while its peer could still signal it.
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  // A wait that ran out in one CTA: all of its cluster wind down with it, as what is in
  // flight may be theirs. (The producer may have ended before: what it issued is waited for
  // here, when no role runs any more.)
  if (*abort_v && threadIdx.x < static_cast<unsigned>(2 * p.parts))
    st_dsmem_u32(map_to_rank(smem_u32(&wind_down), threadIdx.x), 1);
  __syncwarp();
  cluster_sync();
  if (*const_cast<volatile int*>(&wind_down) != 0) {
    if (rank == 1 && threadIdx.x < sizeof(Issued) / 4)
      st_dsmem_u32(map_to_rank(smem_u32(&odd_issued) + threadIdx.x * 4, even),
                   reinterpret_cast<const volatile uint32_t*>(&issued)[threadIdx.x]);
    __syncwarp();
    cluster_sync();
    if (warp == 1 && rank == 0 && elect_one()) {
      // The MMAs issued before the abort: a commit behind them, waited for.
      umma_commit_pair(smem_u32(&drain_bar), 0x1 << even);
      wait_drain(smem_u32(&drain_bar), 0);
    }
    if (threadIdx.x == 0) {
      if (rank == 0) drain_copies(full_bar, stages, issued, odd_issued);
      for (int s = 0; s < stages; ++s)  // the last tail of each stage
        if (issued.tails[s] != 0) wait_drain(smem_u32(&tail_bar[s]), (issued.tails[s] - 1) & 1u);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

typedef void (*Kernel)(const CUtensorMap, const Maps, const Params);

constexpr Kernel kKernels[] = {
    expert_kernel<kGated, kActSilu>, expert_kernel<kGated, kActGelu>,
    expert_kernel<kRows, kActSilu>, expert_kernel<kRowsT, kActSilu>,
    expert_kernel<kWeights, kActSilu>};

int ceil_div(int a, int b) { return (a + b - 1) / b; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Clusters of one to four pairs that are resident at once, by device (its set-up has the
// lock).
constexpr int kMaxDevices = 64;
constexpr int kMaxParts = 4;
int g_clusters[kMaxDevices][kMaxParts];

int resident(const DeviceInfo& dev, int parts) { return g_clusters[dev.device][parts - 1]; }

// How a call is cut: rows (kWeights: columns) of a tile and pairs that share a sum.
struct Cut {
  int tile_rows, parts;
  int64_t tiles;  // at most
};

// Cycles of one tile, and of meeting for a sum, fitted to calls of one to 64 tiles and one to
// three waves (us measured: 1000 rows of 2048 against 2048 weight rows with tiles of 256,
// 128 and 64 rows 16.6, 13.0 and 16.2; 128 rows of 7168, 2 x 2048 weight rows, one to three
// pairs per sum 28.9, 22.7 and 21.5; 64 rows of them 23.3, 18.4 and 17.8). A block of 128
// columns takes about its MMAs' time, four cycles a row, and no less than the weights need
// to come in. It counts neither the bytes of narrower tiles, nor rows that span one line more
// for their pitch, nor a tile's stores, and is too low where these bind: both products of the
// gradient of 777 rows (5128 columns, F = 1000) take 22 us each, by this 13; a tile of the
// weights' gradient of 60 experts of 91 rows 7300 cycles, by this 2800.
int64_t tile_cycles(int blocks, int rows, int parts) {
  const int64_t block = std::max<int64_t>(570, 240 + 21 * rows / 5);
  return ceil_div(blocks, parts) * block + 1500 +
         (parts > 1 ? 2500 + (parts - 1) * (2500 + 20 * rows) : 0);
}

// The stages of a form's tiles of `rows` rows (kWeights: columns).
struct Ring {
  int stages, stage_bytes;
};

// More than the kernels' static shared memory (setup_experts would fail with less).
constexpr int kStaticBytes = 512;

// As many stages as fit beside the chunks, the experts' table and static shared memory: of
// 64 KB three, but two where a gated block keeps its projections in bf16 for more than 297
// experts.
Ring ring_of(Form form, int saved_kind, int rows, int E, const DeviceInfo& dev) {
  const int bytes = form == kWeights
                        ? static_cast<int>(2 * kOperandBytes)
                        : static_cast<int>(kOperandBytes) + (rows / 2 + 31) / 32 * 8192;
  const int rest = dev.max_smem_optin - kStaticBytes - 1024 -
                   kGroups * turn_bytes(form, saved_kind) - experts_table_bytes(E);
  return Ring{std::min(kMaxStages, rest / bytes), bytes};
}

// Whether the stages hold the sums of a tile's other pairs, beside the widest chunks of the
// form: the order of a sum does not depend on what is kept.
bool sums_fit(Form form, int parts, int rows, int E, const DeviceInfo& dev) {
  const Ring ring = ring_of(form, kSavedBf16, rows, E, dev);
  return (parts - 1) * rows * 512 <= ring.stages * ring.stage_bytes;
}

// `tiles(rows)` for tiles of at most `rows` rows. Whole waves count: as many tiles as pairs
// are resident run at once.
template <typename Tiles>
Cut cut(const DeviceInfo& dev, Form form, int E, int blocks, int most_rows, int most_parts,
        Tiles tiles) {
  Cut best{};
  int64_t best_cycles = INT64_MAX;
  for (int rows = std::min(kTileRows, most_rows); rows >= 64 || best_cycles == INT64_MAX;
       rows -= 32)
    for (int parts = 1; parts <= most_parts && parts <= blocks; ++parts) {
      const int64_t n = tiles(rows), at_once = std::max(resident(dev, parts), parts == 1 ? 1 : 0);
      if (parts > 1 && (n > at_once || !sums_fit(form, parts, rows, E, dev))) continue;
      const int64_t waves = ceil_div(n, at_once);
      const int64_t cycles = waves * tile_cycles(blocks, rows, parts);
      if (cycles < best_cycles) {
        best_cycles = cycles;
        best = Cut{rows, parts, n};
      }
    }
  return best;
}

// Most tiles of N rows and E experts in passes of `rows` rows.
int64_t most_row_tiles(int N, int E, int mblocks, int rows) {
  return (static_cast<int64_t>(std::min(N, E)) + N / rows) * mblocks;
}

Cut cut_rows(const DeviceInfo& dev, Form form, const int32_t* offsets, int N, int E, int mblocks,
             int K) {
  const int all = (std::min(N, kTileRows) + 31) & ~31;
  if (offsets == nullptr)  // tiles of one size, as the kernel cuts them
    return cut(dev, form, E, ceil_div(K, kBlockK), all, kMaxParts, [&](int rows) {
      return static_cast<int64_t>(ceil_div(N, rows)) * mblocks;
    });
  // The experts' counts are not known here: full tiles, and several pairs per sum where
  // even the most tiles that there can be leave pairs idle.
  Cut c{all, 1, most_row_tiles(N, E, mblocks, all)};
  for (int parts = 2; parts <= kMaxParts && parts <= ceil_div(K, kBlockK); ++parts)
    if (c.tiles <= resident(dev, parts) && sums_fit(form, parts, all, E, dev)) c.parts = parts;
  return c;
}

cudaError_t launch(Kernel kernel, Form form, const CUtensorMap& a_map, const Maps& b_maps, Params p,
                   const Cut& c, const DeviceInfo& dev, cudaStream_t stream) {
  p.err = dev.err_word;
  p.turn = turn_bytes(form, p.saved_kind);
  p.tile_rows = c.tile_rows;
  p.parts = c.parts;
  const Ring ring = ring_of(form, p.saved_kind, c.tile_rows, p.E, dev);
  p.stages = ring.stages;
  p.stage_bytes = ring.stage_bytes;
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + kGroups * p.turn +
                      experts_table_bytes(p.E);
  const int clusters = static_cast<int>(
      p.parts > 1 ? c.tiles : std::min<int64_t>(std::max(1, resident(dev, 1)), c.tiles));
  return launch_dependent_clusters(2 * p.parts, kernel, dim3(2 * p.parts * clusters),
                                   dim3(kThreads), smem, stream, a_map, b_maps, p);
}

// Whether one copy may bring two 64-column pieces of `cols` columns.
bool whole(int cols) { return cols % 64 == 0; }

// Rows [N, cols] in boxes of 32, 64, 96 and 128 rows, as far as halves of tiles of
// `tile_rows` rows need them.
bool rows_maps(Maps* maps, const void* base, int N, int cols, int tile_rows) {
  for (int i = 0; i < ceil_div(tile_rows / 2, 32); ++i)
    if (!(whole(cols) ? make_map_bf16_rows64(&maps->map[i], base, N, cols, 32 * (i + 1), 2)
                      : make_map_bf16_sw128(&maps->map[i], base, N, cols, 32 * (i + 1))))
      return false;
  return true;
}

// Rows [N, cols] as an MN-major operand: 128 rows deep.
bool sums_map(CUtensorMap* map, const void* base, int N, int cols, bool pieces) {
  return pieces ? make_map_bf16_rows64(map, base, N, cols, 128, 2)
                : make_map_bf16_sw128(map, base, N, cols, 128);
}

// Matrices [E, rows, cols] in boxes of 128 rows of one matrix.
bool matrices_map(CUtensorMap* map, const void* base, int E, int rows, int cols) {
  const uint64_t c = cols, r = rows, n = E;
  if (whole(cols)) {
    const uint64_t dims[] = {64, r, c / 64, n};
    const uint64_t strides[] = {c * 2, 128, r * c * 2};
    const uint32_t box[] = {64, 128, 2, 1};
    return make_map_bf16_nd(map, base, 4, dims, strides, box);
  }
  const uint64_t dims[] = {c, r, n};
  const uint64_t strides[] = {c * 2, r * c * 2};
  const uint32_t box[] = {64, 128, 1};
  return make_map_bf16_nd(map, base, 3, dims, strides, box);
}

// Gate and up rows in turns of eight: (pieces of) columns, 8 rows, gate or up, eights of
// rows of all experts. The eights end F rows before the last row, so that the up rows
// stay within the array; a tile's eights past an expert's F are other rows, whose results
// are not stored.
bool gated_map(CUtensorMap* map, const void* base, int E, int F, int C) {
  const uint64_t c = C, f = F, eights = (2 * static_cast<uint64_t>(E) - 1) * f / 8;
  if (whole(C)) {
    const uint64_t dims[] = {64, 8, 2, eights, c / 64};
    const uint64_t strides[] = {c * 2, f * c * 2, 8 * c * 2, 128};
    const uint32_t box[] = {64, 8, 2, 8, 2};
    return make_map_bf16_nd(map, base, 5, dims, strides, box);
  }
  const uint64_t dims[] = {c, 8, 2, eights};
  const uint64_t strides[] = {c * 2, f * c * 2, 8 * c * 2};
  const uint32_t box[] = {64, 8, 2, 8};
  return make_map_bf16_nd(map, base, 4, dims, strides, box);
}

}  // namespace

cudaError_t setup_experts(const DeviceInfo& dev) {
  for (Kernel k : kKernels) {
    const cudaError_t e = cudaFuncSetAttribute(
        reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize,
        dev.max_smem_optin - kStaticBytes);
    if (e != cudaSuccess) return e;
  }
  // (clusters of several pairs do not always fill every SM: the parts of the GPU that a
  // cluster has to lie in do not all have a multiple of its size)
  for (int i = 0; i < kMaxParts; ++i) {
    const unsigned ctas = 2u * (i + 1);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms) / ctas * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(dev.max_smem_optin) - kStaticBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kKernels[2], &cfg);
    if (e != cudaSuccess) return e;
    g_clusters[dev.device][i] = std::min(n, dev.num_sms / static_cast<int>(ctas));
  }
  return cudaSuccess;
}

cudaError_t launch_expert_gated(const ExpertGatedArgs& a, const DeviceInfo& dev,
                                cudaStream_t stream) {
  if (few_rows(a.offsets, a.N, a.E, a.F, a.C, true, dev)) return launch_expert_gated_few(a, stream);
  Params p{};
  p.offsets = a.offsets;
  p.out = a.hidden;
  p.saved = a.saved;
  p.exponents = a.exponents;
  p.N = a.N;
  p.E = a.E;
  p.M = a.F;
  p.K = a.C;
  p.mblocks = ceil_div(a.F, 128);
  p.saved_kind = a.saved_kind;
  p.ring = a.ring;
  p.whole_a = p.whole_b = whole(a.C);
  const Cut c = cut_rows(dev, kGated, a.offsets, a.N, a.E, p.mblocks, a.C);
  CUtensorMap w_map;
  Maps x_maps{};
  if (!gated_map(&w_map, a.weights, a.E, a.F, a.C) ||
      !rows_maps(&x_maps, a.x, a.N, a.C, c.tile_rows))
    return cudaErrorInvalidValue;
  return launch(kKernels[a.act == kActSilu ? 0 : 1], kGated, w_map, x_maps, p, c, dev, stream);
}

cudaError_t launch_expert_rows(const ExpertRowsArgs& a, const DeviceInfo& dev,
                               cudaStream_t stream) {
  if (!a.transposed && few_rows(a.offsets, a.N, a.E, a.M, a.K, false, dev))
    return launch_expert_rows_few(a, stream);
  Params p{};
  p.offsets = a.offsets;
  p.out = a.out;
  p.N = a.N;
  p.E = a.E;
  p.M = a.M;
  p.K = a.K;
  p.mblocks = ceil_div(a.M, 256);
  p.ring = a.ring;
  p.whole_a = whole(a.transposed ? a.M : a.K);
  p.whole_b = whole(a.K);
  const Form form = a.transposed ? kRowsT : kRows;
  const Cut c = cut_rows(dev, form, a.offsets, a.N, a.E, p.mblocks, a.K);
  CUtensorMap w_map;
  Maps x_maps{};
  if (!(a.transposed ? matrices_map(&w_map, a.weights, a.E, a.K, a.M)
                     : matrices_map(&w_map, a.weights, a.E, a.M, a.K)) ||
      !rows_maps(&x_maps, a.x, a.N, a.K, c.tile_rows))
    return cudaErrorInvalidValue;
  return launch(kKernels[a.transposed ? 3 : 2], form, w_map, x_maps, p, c, dev,
                stream);
}

cudaError_t launch_expert_weights(const ExpertWeightsArgs& a, const DeviceInfo& dev,
                                  cudaStream_t stream) {
  Params p{};
  p.offsets = a.offsets;
  p.out = a.grad_weights;
  p.N = a.N;
  p.E = a.E;
  p.M = a.M;
  p.K = a.C;
  p.mblocks = ceil_div(a.M, 256);
  const int mean = ceil_div(a.N, a.E);
  const int most_parts = a.offsets == nullptr ? kMaxParts : 1;  // (of blocks known here)
  const Cut c = cut(dev, kWeights, a.E, ceil_div(mean, kBlockK), (a.C + 31) & ~31, most_parts,
                    [&](int cols) {
                      return static_cast<int64_t>(a.E) * p.mblocks * ceil_div(a.C, cols);
                    });
  p.cblocks = ceil_div(a.C, c.tile_rows);
  p.ring = a.ring;
  p.whole_a = whole(a.M);
  p.whole_b = whole(a.C) && c.tile_rows % 128 == 0;  // (a half begins at a whole piece)
  CUtensorMap g_map;
  Maps x_maps{};
  if (!sums_map(&g_map, a.grad, a.N, a.M, p.whole_a) ||
      !sums_map(&x_maps.map[0], a.x, a.N, a.C, p.whole_b))
    return cudaErrorInvalidValue;
  return launch(kKernels[4], kWeights, g_map, x_maps, p, c, dev, stream);
}

}  // namespace lt
