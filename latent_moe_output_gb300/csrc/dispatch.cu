// latent_tail_dispatch: a stable sort of the router's T * K choices by expert,
// and a copy of each token's row to its choices' places.
//
// A choice i has key(i) = its expert, or E without one, and the place
//   row(i) = #{j : key(j) < key(i)} + #{j < i : key(j) == key(i)}.
//
// Up to kDispatchOneLaunch choices, one kernel with one CTA per choice counts
// that definition directly over all ids (a few loads per thread, from L2) while its
// row is on its way, and copies the row: one launch, no workspace (2.0 us at 128
// choices, of which nothing but latency is left).
// Above that the choices are cut into contiguous chunks, one CTA each: a first
// kernel counts the experts of each chunk; a second sums the counts of the chunks
// before its own (so every CTA knows where its choices of each expert begin), ranks
// its own choices with warp-wide matches, and copies their rows, or leaves that to a
// third kernel that reads each row of x once for all its places. Memory bounds the
// copy: 131072 choices of 16384 tokens, L = 2048: 98.5 us for 604 MB, 6.1 TB/s, 90 % of
// the measured copy rate, with 88 us for the copy and the rest for the sort. (Bringing x
// into L2 during the sort did not help: the writes of the call before still drain
// then.) No atomics decide an order: the places are the same from run to run.
#include "block_launch.h"
#include "rows.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kSmallThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxChunk = 65535;
static_assert(static_cast<int64_t>(kDispatchMaxChunks) * kMaxChunk >= kMaxSlots, "16-bit counts");
constexpr int kCopyThreads = 256;
// The ranking kernel copies its chunk's rows itself up to this size, above it a third
// kernel does (measured with 8 choices of 256 experts, L = 2048, us with two and three
// kernels: T = 512 8.2 and 11.3, 1024 11.5 and 13.0, 2048 18.0 and 18.7, 4096 32.3 and
// 30.8), and for rows of less than a warp's 16-byte pieces up to kMaxNarrowRows choices
// per chunk (8 choices, L = 72: T = 605 5.9 and 7.1, 4000 8.3 and 7.2).
constexpr size_t kMaxFusedBytes = size_t(80) << 20;
constexpr int kMaxNarrowRows = 128;
constexpr int kMaxChunkRows = 4096;  // choices per chunk that the ranking kernel copies itself

__device__ __forceinline__ int choice_key(int id, int E) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(E) ? id : E;
}

__global__ void __launch_bounds__(kSmallThreads)
    dispatch_small_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids,
                          uint16_t* __restrict__ rows, int32_t* __restrict__ offsets,
                          int32_t* __restrict__ order, int32_t* __restrict__ position, int n,
                          int K, int E, int nch) {
  __shared__ int s_rank[kSmallThreads / 32], s_prev[kSmallThreads / 32],
      s_same[kSmallThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int key = choice_key(ids[i], E);
  const uint4* src = reinterpret_cast<const uint4*>(x) + static_cast<size_t>(i / K) * nch;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (key < E && tid < nch) v = ld_stream_v4(src + tid);

  int rank = 0, prev = 0, same = 0;  // prev: 1 + largest key below this one
  for (int j = tid; j < n; j += kSmallThreads) {
    const int kj = choice_key(ids[j], E);
    if (kj < key) {
      ++rank;
      prev = max(prev, kj + 1);
    } else if (kj == key && j < i) {
      ++same;
    }
  }
  rank = __reduce_add_sync(0xffffffffu, rank);
  prev = __reduce_max_sync(0xffffffffu, prev);
  same = __reduce_add_sync(0xffffffffu, same);
  if ((tid & 31) == 0) {
    s_rank[tid >> 5] = rank;
    s_prev[tid >> 5] = prev;
    s_same[tid >> 5] = same;
  }
  __syncthreads();
  rank = prev = same = 0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / 32; ++w) {
    rank += s_rank[w];
    prev = max(prev, s_prev[w]);
    same += s_same[w];
  }
  const int below = rank;
  rank += same;

  if (tid == 0) {
    order[rank] = i;
    position[i] = key < E ? rank : ~rank;
  }
  if (same == 0)  // first choice of its key: it opens this key and the empty ones before it
    for (int e = prev + tid; e <= key; e += kSmallThreads) offsets[e] = below;
  if (rank == n - 1)  // last choice: it closes the keys above its own
    for (int e = key + 1 + tid; e <= E; e += kSmallThreads) offsets[e] = n;
  uint4* dst = reinterpret_cast<uint4*>(rows) + static_cast<size_t>(rank) * nch;
  if (tid < nch) dst[tid] = v;
  for (int c = tid + kSmallThreads; c < nch; c += kSmallThreads)
    dst[c] = key < E ? ld_stream_v4(src + c) : make_uint4(0, 0, 0, 0);
}

// Chunk b holds choices [b * per_chunk, min(n, (b + 1) * per_chunk)).
__global__ void __launch_bounds__(kSortThreads)
    dispatch_count_kernel(const int32_t* __restrict__ ids, uint16_t* __restrict__ counts, int n,
                          int E, int per_chunk, int stride) {
  extern __shared__ uint32_t s_count[];  // [stride]
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < stride; e += kSortThreads) s_count[e] = 0;
  __syncthreads();
  pdl_wait();
  const int lo = blockIdx.x * per_chunk, hi = min(n, lo + per_chunk);
  for (int i = lo + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&s_count[choice_key(ids[i], E)], 1u);
  __syncthreads();
  uint16_t* out = counts + static_cast<size_t>(blockIdx.x) * stride;
  for (int e = threadIdx.x; e < stride; e += kSortThreads)
    out[e] = static_cast<uint16_t>(s_count[e]);
}

__global__ void __launch_bounds__(kSortThreads)
    dispatch_rank_kernel(const int32_t* __restrict__ ids, const uint16_t* __restrict__ counts,
                         int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                         int32_t* __restrict__ position, int n, int E, int per_chunk, int stride,
                         const uint16_t* __restrict__ x, uint16_t* __restrict__ rows, int K,
                         int nch) {
  extern __shared__ uint32_t smem[];
  uint32_t* s_before = smem;           // [stride] choices of the expert in earlier chunks
  uint32_t* s_total = smem + stride;   // [stride] choices of the expert in all chunks
  uint16_t* s_warp = reinterpret_cast<uint16_t*>(smem + 2 * stride);  // [warps][stride]
  int32_t* s_place = reinterpret_cast<int32_t*>(s_warp + kSortWarps * stride);  // with nch != 0
  __shared__ uint32_t s_scan[kSortWarps];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < stride; e += kSortThreads) s_before[e] = s_total[e] = 0;
  uint32_t* z = reinterpret_cast<uint32_t*>(s_warp);
  for (int e = tid; e < kSortWarps * stride / 2; e += kSortThreads) z[e] = 0;
  __syncthreads();
  pdl_wait();

  // Counts of all chunks, eight experts (16 bytes) per thread and load.
  const int nvec = stride / 8, slices = kSortThreads / nvec;
  const int vec = tid % nvec, slice = tid / nvec;
  if (slice < slices) {
    uint32_t tot[8] = {}, bef[8] = {};
    for (int b = slice; b < static_cast<int>(gridDim.x); b += slices) {
      const uint4 v = *reinterpret_cast<const uint4*>(counts + static_cast<size_t>(b) * stride +
                                                      vec * 8);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      const bool earlier = b < static_cast<int>(blockIdx.x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t c = (w[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        tot[j] += c;
        if (earlier) bef[j] += c;
      }
    }
    // (element j of all vectors side by side, so that a warp's atomics meet 32 banks)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (tot[j]) atomicAdd(&s_total[j * nvec + vec], tot[j]);
      if (bef[j]) atomicAdd(&s_before[j * nvec + vec], bef[j]);
    }
  }
  // Each warp counts its own contiguous part of the chunk.
  const int lo = blockIdx.x * per_chunk, hi = min(n, lo + per_chunk);
  const int per_warp = ((per_chunk + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int wlo = min(hi, lo + warp * per_warp), whi = min(hi, wlo + per_warp);
  uint16_t* mine = s_warp + warp * stride;
  for (int base = wlo; base < whi; base += 32) {
    const int i = base + lane;
    const int key = i < whi ? choice_key(ids[i], E) : -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && lane == __ffs(peers) - 1)
      mine[key] = static_cast<uint16_t>(mine[key] + __popc(peers));
    __syncwarp();
  }
  __syncthreads();

  // First place of every expert: an exclusive sum over the experts (at most one
  // per thread); the choices without an expert begin after the last one.
  auto at = [&](int e) { return (e & 7) * nvec + (e >> 3); };
  const uint32_t own = tid < E ? s_total[at(tid)] : 0;
  uint32_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    uint32_t v = s_scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += up;
    }
    s_scan[lane] = v;
  }
  __syncthreads();
  const uint32_t first = incl - own + (warp > 0 ? s_scan[warp - 1] : 0);
  const uint32_t routed = s_scan[kSortWarps - 1];
  if (tid < E) {
    s_before[at(tid)] += first;
    if (blockIdx.x == 0) offsets[tid] = static_cast<int32_t>(first);
  }
  if (tid == 0) {
    s_before[at(E)] += routed;
    if (blockIdx.x == 0) offsets[E] = static_cast<int32_t>(routed);
  }
  for (int e = tid; e <= E; e += kSortThreads) {  // exclusive sum over the warps
    uint32_t run = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = s_warp[w * stride + e];
      s_warp[w * stride + e] = static_cast<uint16_t>(run);
      run += c;
    }
  }
  __syncthreads();

  for (int base = wlo; base < whi; base += 32) {
    const int i = base + lane;
    const int key = i < whi ? choice_key(ids[i], E) : -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    const uint32_t before = key >= 0 ? mine[key] : 0;
    __syncwarp();
    if (key >= 0) {
      const int row = static_cast<int>(s_before[at(key)] + before +
                                       __popc(peers & ((1u << lane) - 1)));
      order[row] = i;
      position[i] = key < E ? row : ~row;
      if (nch != 0) s_place[i - lo] = key < E ? row : ~row;
      if (lane == __ffs(peers) - 1)
        mine[key] = static_cast<uint16_t>(before + __popc(peers));
    }
    __syncwarp();
  }
  if (nch == 0) return;
  // The chunk's rows, one choice per warp at a time (x comes from L2 after the first).
  __syncthreads();
  const uint4* x4 = reinterpret_cast<const uint4*>(x);
  uint4* r4 = reinterpret_cast<uint4*>(rows);
  for (int i = lo + warp; i < hi; i += kSortWarps) {
    const int p = s_place[i - lo];
    const uint4* src = x4 + static_cast<size_t>(i / K) * nch;
    uint4* dst = r4 + static_cast<size_t>(p >= 0 ? p : ~p) * nch;
#pragma unroll 4
    for (int c = lane; c < nch; c += 32)
      st_stream_v4(dst + c, p >= 0 ? src[c] : make_uint4(0, 0, 0, 0));
  }
}

// One thread per 16-byte piece of x: read once, written to the K places.
__global__ void __launch_bounds__(kCopyThreads)
    dispatch_copy_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ position,
                         uint16_t* __restrict__ rows, int T, int K, int nch) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kCopyThreads;
  const int t0 = static_cast<int>(base / nch);
  const int rem = static_cast<int>(base - static_cast<int64_t>(t0) * nch) + threadIdx.x;
  const int t = t0 + rem / nch, c = rem % nch;
  if (t >= T) return;
  const uint4 v = ld_stream_v4(reinterpret_cast<const uint4*>(x) + static_cast<size_t>(t) * nch + c);
  const int32_t* pos = position + static_cast<size_t>(t) * K;
  uint4* dst = reinterpret_cast<uint4*>(rows) + c;
  const int n = T * K;
  for (int k = 0; k < K; ++k) {
    const int p = pos[k];
    const int row = p >= 0 ? p : ~p;
    if (row < n)
      st_stream_v4(dst + static_cast<size_t>(row) * nch, p >= 0 ? v : make_uint4(0, 0, 0, 0));
  }
}

size_t rank_smem(int stride) {
  return static_cast<size_t>(stride) * (2 * sizeof(uint32_t) + kSortWarps * sizeof(uint16_t));
}

}  // namespace

cudaError_t setup_dispatch(const DeviceInfo&) {
  return cudaFuncSetAttribute(dispatch_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(rank_smem(dispatch_counts_stride(kMaxExperts)) +
                                               kMaxChunkRows * sizeof(int32_t)));
}

cudaError_t launch_dispatch(const DispatchArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int n = a.T * a.K;
  const int nch = a.rows != nullptr ? a.L / 8 : 0;
  if (n <= kDispatchOneLaunch)
    return launch_dependent(dispatch_small_kernel, dim3(n), dim3(kSmallThreads), 0, stream, a.x,
                            a.ids, a.rows, a.offsets, a.order, a.position, n, a.K, a.E, nch);
  const int stride = dispatch_counts_stride(a.E);
  // One chunk per SM, more where a chunk would not fit its 16-bit counts.
  const int chunks = std::min(kDispatchMaxChunks,
                              std::max(dev.num_sms, (n + kMaxChunk - 1) / kMaxChunk));
  const int per_chunk = (n + chunks - 1) / chunks;
  cudaError_t e = launch_dependent(dispatch_count_kernel, dim3(chunks), dim3(kSortThreads),
                                   stride * sizeof(uint32_t), stream, a.ids, a.counts, n, a.E,
                                   per_chunk, stride);
  if (e != cudaSuccess) return e;
  const bool fused = nch != 0 && per_chunk <= kMaxChunkRows &&
                     (nch >= 32 || per_chunk <= kMaxNarrowRows) &&
                     static_cast<size_t>(n) * a.L * 2 <= kMaxFusedBytes;
  e = launch_dependent(dispatch_rank_kernel, dim3(chunks), dim3(kSortThreads),
                       rank_smem(stride) + (fused ? per_chunk * sizeof(int32_t) : 0), stream,
                       a.ids, static_cast<const uint16_t*>(a.counts), a.offsets, a.order,
                       a.position, n, a.E, per_chunk, stride, a.x, a.rows, a.K, fused ? nch : 0);
  if (e != cudaSuccess || nch == 0 || fused) return e;
  const int64_t pieces = static_cast<int64_t>(a.T) * nch;
  return launch_dependent(dispatch_copy_kernel,
                          dim3(static_cast<unsigned>((pieces + kCopyThreads - 1) / kCopyThreads)),
                          dim3(kCopyThreads), 0, stream, a.x,
                          static_cast<const int32_t*>(a.position), a.rows, a.T, a.K, nch);
}

}  // namespace lt
