/*
 * latent_tail.h - C ABI of the GB300 (sm_103a) latent-MoE output tail.
 *
 * The operation (Kimi-K3 latent MoE, as the vLLM PR #50383 and #51253 digests
 * describe it):
 *
 *   x[t,l]   = sum_{p<P} routed[p,t,l]                      routed partial sum
 *   y[t,l]   = x[t,l] * rsqrt(mean_l x[t,l]^2 + eps) * g[l]  RMSNorm with weight
 *   out[t,h] = sum_l y[t,l] * W[h,l] + sum_{p<P} shared[p,t,h]
 *
 * Sources, by page and section:
 *   - PR #51253 report, test source section: `_check_matches_replicated`
 *     (expected = F.linear(F.rms_norm(all-reduced routed, (L,), g, EPS), W)
 *     plus the all-reduced shared output) and `_check_writes_only_its_own_shard`
 *     (a rank owning columns [start,end) adds latent . W[start:end]^T into only
 *     those columns; the rest stays bit-identical).
 *   - PR #50383 report, source of `_shard_up_proj_tail`: all-reduce then norm
 *     (`allreduce_norm_latent_out`), `weight.narrow(0, start, size)` and
 *     `shared_output.narrow(-1, start, size)`, then the beta-add epilogue
 *     `hidden_shard.addmm_(latent, up_proj_shard.t())`.
 *   On one GPU the P tensor-parallel partials are stacked tensors that the
 *   kernels reduce; the column-parallel shard is the [col_start, col_end) option.
 *
 * Conventions for every entry point:
 *   - bf16 tensors are passed as `uint16_t*` holding bfloat16 bit patterns.
 *   - All arrays are DEVICE memory on the current CUDA device (except the
 *     host buffers of latent_tail_forward_host), contiguous and row-major,
 *     allocated and owned by the caller. Every pointer must be
 *     16-byte aligned. The library never allocates, frees or keeps a pointer
 *     after the call returns.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream). No call synchronizes the host, except
 *     latent_tail_check.
 *   - Arguments are validated on the host before anything is enqueued. On a
 *     non-OK status nothing was launched and no memory was touched.
 *   - T == 0 is a no-op that returns LT_OK.
 *   - Shape limits: 1 <= P <= 64; 8 <= L <= 16384 and L % 8 == 0;
 *     8 <= H <= 1048576 and H % 8 == 0; 0 <= T <= 2^24. Violations give
 *     LT_ERR_INVALID_ARG (range) or LT_ERR_ALIGNMENT (multiple of 8).
 *   - Device-side waits are bounded: a wait that expires sets a device error
 *     word and the kernel returns early; latent_tail_check reports it as
 *     LT_ERR_TIMEOUT.
 */
#ifndef LATENT_TAIL_H
#define LATENT_TAIL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define LT_API __attribute__((visibility("default")))
#else
#define LT_API
#endif

typedef enum lt_status {
  LT_OK = 0,
  LT_ERR_INVALID_ARG = 1, /* null pointer, bad shape/range, overlap, bad eps */
  LT_ERR_ALIGNMENT = 2,   /* pointer not 16-byte aligned, or L/H/range not % 8 */
  LT_ERR_UNSUPPORTED = 3, /* current device is not compute capability 10.3 */
  LT_ERR_WORKSPACE = 4,   /* workspace missing or smaller than required */
  LT_ERR_CUDA = 5,        /* a CUDA runtime call or kernel launch failed */
  LT_ERR_TIMEOUT = 6      /* a bounded device-side wait expired */
} lt_status;

/* Same object as cudaStream_t. */
typedef struct CUstream_st* lt_stream;

/*
 * Bytes of device workspace latent_tail_forward / _forward_cols need for T
 * tokens of latent width L: the normalized latent y [T, L] in bf16, rounded up
 * to 256 bytes. P and H do not change it. Returns 0 for T <= 0 or invalid
 * shapes. Host-only, never touches the GPU.
 */
LT_API size_t latent_tail_workspace_size(int P, int T, int L, int H);

/*
 * Whole tail for all H output columns (equivalent to latent_tail_forward_cols
 * with col_start = 0, col_end = H).
 *   routed      [P, T, L] bf16  routed-expert latent partials
 *   shared      [P, T, H] bf16  shared-expert output partials
 *   norm_weight [L]       fp32  RMSNorm weight g, or NULL for the pages'
 *                               `transform.norm is None` branch: no RMSNorm, the
 *                               latent is the partial sum itself (eps unused)
 *   W           [H, L]    bf16  up-projection weight (row h = output column h)
 *   out         [T, H]    bf16  result, round-to-nearest-even; must not overlap
 *                               routed, W, g or the workspace. It may be exactly
 *                               one of the shared partials (out == shared + p*T*H):
 *                               the pages' in-place `addmm_` into the shared
 *                               output; any other overlap with shared is rejected
 *   eps                         RMSNorm epsilon, finite and > 0 (when norm_weight
 *                               is not NULL)
 *   workspace, workspace_bytes  at least latent_tail_workspace_size(P,T,L,H)
 *                               bytes of device scratch; its contents on entry
 *                               are ignored and on return are unspecified
 * For T <= 2 (when L <= 4096 and one SM's share of W fits in its shared
 * memory, e.g. L = 2048 at H = 7168) one CUDA-core kernel does the whole tail;
 * the normalized latent then stays in FP32, unrounded, and the workspace is
 * not used. Otherwise two kernels run: reduce + RMSNorm into the workspace
 * (bf16), then the up-projection with the shared-partial epilogue (decode
 * kernel for T <= 224 when its buffers fit in shared memory, which they always
 * do for T <= 128 and do at L = 2048; persistent tensor-core kernel otherwise),
 * chained by programmatic dependent launch. When the decode kernel runs (and
 * T > 2) the first kernel also prefetches routed and the W rows
 * into L2 before it waits for the preceding work on the stream (an L2
 * prefetch is only a hint: if that work is still writing routed, the lines are
 * updated in L2 and every read happens after the wait). Calls issued back to
 * back on one stream may share one workspace. Capturable in a CUDA graph.
 */
LT_API lt_status latent_tail_forward(const uint16_t* routed, const uint16_t* shared,
                                     const float* norm_weight, const uint16_t* W,
                                     uint16_t* out, int P, int T, int L, int H,
                                     float eps, void* workspace, size_t workspace_bytes,
                                     lt_stream stream);

/*
 * Column-parallel form: writes only out[t, h] for col_start <= h < col_end.
 * Every other byte of out (still the full [T, H] buffer) is left untouched.
 * 0 <= col_start < col_end <= H, both multiples of 8. Each written element is
 * computed exactly as latent_tail_forward computes it, so a set of calls whose
 * ranges tile [0, H) reproduces the full call bit for bit.
 */
LT_API lt_status latent_tail_forward_cols(const uint16_t* routed, const uint16_t* shared,
                                          const float* norm_weight, const uint16_t* W,
                                          uint16_t* out, int P, int T, int L, int H,
                                          float eps, int col_start, int col_end,
                                          void* workspace, size_t workspace_bytes,
                                          lt_stream stream);

/*
 * Steps 1-2 alone (the pages' `allreduce_norm_latent_out`): latent[t,l] =
 * bf16_rn(x[t,l] * rsqrt(mean_l x^2 + eps) * g[l]) with x = sum_p routed[p,t,l]
 * accumulated in FP32; with norm_weight == NULL, latent = bf16_rn(x).
 *   routed [P, T, L] bf16, norm_weight [L] fp32, latent [T, L] bf16 (output,
 *   must not overlap the inputs).
 */
LT_API lt_status latent_tail_norm(const uint16_t* routed, const float* norm_weight,
                                  uint16_t* latent, int P, int T, int L, float eps,
                                  lt_stream stream);

/*
 * Steps 3-5 alone (the pages' narrowed `addmm_` beta-add plus the shared-partial
 * sum): out[t,h] = bf16_rn(sum_l latent[t,l] * W[h,l] + sum_p shared[p,t,h]) for
 * col_start <= h < col_end; other columns untouched.
 *   latent [T, L] bf16, shared [P, T, H] bf16, W [H, L] bf16, out [T, H] bf16
 *   (out may be exactly one of the shared partials, as in latent_tail_forward).
 * Range rules as in latent_tail_forward_cols; results are bit-identical to the
 * projection step of latent_tail_forward given the same latent. With P = 1 this
 * is the per-rank compute after the reference's all-reduce.
 * When the decode kernel serves the call (see latent_tail_forward) it is
 * launched as a programmatic dependent of the work
 * before it on the stream: it may start (set up its barriers and tensor memory)
 * before that work has finished, but it reads no input and writes no output
 * until that work is complete, so back-to-back calls overlap only set-up.
 */
LT_API lt_status latent_tail_project_cols(const uint16_t* latent, const uint16_t* shared,
                                          const uint16_t* W, uint16_t* out, int P, int T,
                                          int L, int H, int col_start, int col_end,
                                          lt_stream stream);

/*
 * Synchronizes `stream`, then reports (and clears) the current device's error
 * word: LT_ERR_TIMEOUT if a bounded device wait expired since the last check,
 * LT_ERR_CUDA if the stream reported an error, LT_OK otherwise.
 */
LT_API lt_status latent_tail_check(lt_stream stream);

/*
 * Diagnostic for the bounded device waits: enqueues one CTA that waits on a
 * barrier nothing ever completes, through the same bounded wait the kernels
 * use, with a limit of limit_us microseconds (1 .. 1000000). The wait expires,
 * the device error word records a timeout and the kernel returns; the next
 * latent_tail_check on the stream reports LT_ERR_TIMEOUT and clears it. No
 * fault, trap or hang is involved and the context stays usable.
 */
LT_API lt_status latent_tail_selftest_wait_timeout(unsigned int limit_us, lt_stream stream);

/*
 * Allocation-free form of latent_tail_forward (the pages have no counterpart;
 * this exists for callers, not for the method). Some callers cannot allocate
 * device memory: a custom op or plugin that a host runtime hands only its
 * input and output buffers, with no allocator to call, or code that must not
 * allocate while it runs. They cannot supply the workspace that
 * latent_tail_forward needs, so this entry point keeps that scratch (the
 * normalized latent, T * L * 2 bytes) in a fixed device array inside the
 * library instead:
 *   - the array holds LT_NOALLOC_MAX_SCRATCH_BYTES (8 MiB) on every GPU that
 *     loads the library, until the process exits; calls whose
 *     latent_tail_workspace_size(P, T, L, H) exceeds it return LT_ERR_WORKSPACE
 *     and launch nothing (at L = 2048 that allows T <= 2048);
 *   - nothing is allocated or freed by the call (no cudaMalloc / cudaFree);
 *   - the first call on a device looks up the array's device address on that
 *     device; make that first call before capturing a stream into a graph;
 *   - all calls on a device share the one array and it keeps the previous
 *     call's contents (every call rewrites all of the latent it reads, so
 *     nothing needs to start at zero).
 *     Calls whose GPU work overlaps in time
 *     (different streams without ordering, or different host threads) race on
 *     the array and give wrong results: order them on one stream.
 * Arguments, output and errors are as for latent_tail_forward, minus the
 * workspace.
 */
#define LT_NOALLOC_MAX_SCRATCH_BYTES ((size_t)8 << 20)
LT_API lt_status latent_tail_forward_noalloc(const uint16_t* routed, const uint16_t* shared,
                                             const float* norm_weight, const uint16_t* W,
                                             uint16_t* out, int P, int T, int L, int H,
                                             float eps, lt_stream stream);

/*
 * Bytes of device workspace latent_tail_forward_host needs: the normalized
 * latent as for latent_tail_workspace_size, plus device staging for routed when
 * T <= 2, and for routed, shared and out when the call runs the persistent
 * tensor-core kernel (above 224 tokens, or above 128 when the decode kernel's
 * buffers do not fit; see latent_tail_forward), each rounded up to 256 bytes.
 * Returns 0 for T <= 0 or invalid shapes. Host-only, never touches the GPU.
 */
LT_API size_t latent_tail_host_workspace_size(int P, int T, int L, int H);

/*
 * End-to-end form of latent_tail_forward for inputs that arrive in, and a
 * result that leaves to, host memory (serving glue that holds the partials on
 * the CPU side; the pages' tail always runs on device tensors, so this is a
 * library convenience, not a step of the method).
 *   routed_host [P, T, L], shared_host [P, T, H], out_host [T, H]: bf16 in
 *     PAGE-LOCKED host memory mapped for the current device (cudaHostAlloc /
 *     cudaMallocHost, or cudaHostRegister with cudaHostRegisterMapped), each
 *     lying inside one such allocation, 16-byte aligned. Anything else
 *     (pageable memory, device memory, a range running past its allocation)
 *     gives LT_ERR_INVALID_ARG before any work is enqueued.
 *   norm_weight, W: device memory, as in latent_tail_forward.
 *   out_host: same overlap rules as out in latent_tail_forward (it may be
 *     exactly one of the shared partials).
 *   workspace: latent_tail_host_workspace_size(P, T, L, H) bytes of device
 *     memory, not overlapping W or norm_weight.
 * When the one-launch kernel serves the shape (T <= 2, as for
 * latent_tail_forward), a copy kernel first brings the routed partials into
 * the workspace; the kernel then reads shared and writes out through the host
 * link. Otherwise, when the decode kernel serves the call, the kernels read the
 * partials and write the result through the host link directly: no staging
 * copy, the host bytes cross the link once.
 * For the persistent kernel the partials are copied into the workspace (one cudaMemcpyAsync per
 * tensor), the device path runs, and the result is copied back. Like every
 * call it is asynchronous: out_host holds the result once `stream` has been
 * synchronized, and the host buffers must not be modified before then.
 * Results are bit-identical to latent_tail_forward on the same values.
 */
LT_API lt_status latent_tail_forward_host(const uint16_t* routed_host,
                                          const uint16_t* shared_host,
                                          const float* norm_weight, const uint16_t* W,
                                          uint16_t* out_host, int P, int T, int L, int H,
                                          float eps, void* workspace, size_t workspace_bytes,
                                          lt_stream stream);

/*
 * ---------------------------------------------------------------------------
 * Operators around the tail in a latent-MoE block. The tail turns the experts'
 * latent outputs into the block's output; these produce its routed operand and
 * consume its result:
 *
 *   latent tokens -> latent_tail_dispatch -> experts (latent_tail_expert_matvec4)
 *     -> latent_tail_combine -> routed partial -> latent_tail_forward
 *     -> latent_tail_residual_norm -> the next block
 *
 * The conventions at the top of this file hold (device arrays, contiguous,
 * 16-byte aligned, caller-owned, nothing launched on a non-OK status, outputs
 * must not overlap inputs or one another unless stated). Arrays that a device
 * kernel indexes by (expert ids, positions, offsets) are bounds-checked on the
 * device: a value out of range never leads to an access out of range. Results
 * are the same bits from run to run.
 * After a wait that expired (LT_ERR_TIMEOUT) outputs are incomplete: an element with a
 * token index, of an in-place residual too, is the call's result or untouched; gradients
 * summed over tokens lack tokens.
 */

/*
 * Bytes of device workspace latent_tail_dispatch needs for T tokens with K
 * choices among E experts: 0 where one kernel does the whole call (up to 2048
 * choices), else the per-chunk expert counts. Returns 0 for T <= 0 or invalid
 * shapes. Host-only.
 */
LT_API size_t latent_tail_dispatch_workspace_size(int T, int K, int E);

/*
 * Sorts the T * K choices of an expert router by expert and copies each token's
 * row to its choices' places. With i = t * K + k the flat index of a choice,
 * key(i) = ids[i] where 0 <= ids[i] < E and E otherwise (no expert: the choice
 * is not routed), and row(i) the place of i when the choices are ordered by key
 * and, within one key, by i:
 *   order[row(i)]  = i
 *   position[i]    = row(i) if routed, else -1 - row(i)
 *   offsets[e]     = number of choices with key < e, e = 0 .. E (expert e owns
 *                    rows offsets[e] .. offsets[e+1] - 1; offsets[E] rows in all)
 *   rows[row(i),:] = x[t,:] if routed, else zero (the rows past offsets[E])
 *   x [T, L] bf16, expert_ids [T, K] int32; rows [T*K, L] bf16, offsets [E+1],
 *   order [T*K], position [T, K] int32 (outputs). x and rows may both be NULL:
 *   the sort alone (L is then ignored).
 * Limits: 1 <= K <= 64, 1 <= E <= 1024, T * K <= 2^24, L as for the tail.
 * With T == 0 only offsets is written (zeros).
 * The gradient of x is latent_tail_combine of the rows' gradients without weights.
 */
LT_API lt_status latent_tail_dispatch(const uint16_t* x, const int32_t* expert_ids,
                                      uint16_t* rows, int32_t* offsets, int32_t* order,
                                      int32_t* position, int T, int K, int E, int L,
                                      void* workspace, size_t workspace_bytes,
                                      lt_stream stream);

/*
 * Brings rows sorted by expert back to their tokens: out[t,:] = sum over the
 * routed choices k, ascending, of weights[t,k] * rows[position[t,k],:] (FP32,
 * rounded once to bf16). Choices with position outside [0, T*K) are skipped
 * (their weights are not read into the sum); a token without a routed choice
 * gives zeros.
 *   rows [T*K, L] bf16, position [T, K] int32, weights [T, K] fp32 or NULL
 *   (all 1), out [T, L] bf16 (e.g. one plane of the tail's routed operand).
 */
LT_API lt_status latent_tail_combine(const uint16_t* rows, const int32_t* position,
                                     const float* weights, uint16_t* out, int T, int K, int L,
                                     lt_stream stream);

/*
 * Gradient of latent_tail_combine: for each routed choice, with r = position[t,k],
 *   grad_rows[r,:]    = weights[t,k] * grad_out[t,:]
 *   grad_weights[t,k] = sum_l grad_out[t,l] * rows[r,l]      (FP32)
 * and for each choice that is not routed (position = -1 - r, as
 * latent_tail_dispatch writes it) grad_rows[r,:] = 0 and grad_weights[t,k] = 0.
 * Every row of grad_rows is written when position comes from latent_tail_dispatch.
 *   grad_out [T, L] bf16, rows [T*K, L] bf16, position [T, K], weights [T, K] fp32
 *   or NULL (all 1); grad_rows [T*K, L] bf16, grad_weights [T, K] fp32 or NULL
 *   (not wanted; rows is then not read and may be NULL too).
 */
LT_API lt_status latent_tail_combine_backward(const uint16_t* grad_out, const uint16_t* rows,
                                              const int32_t* position, const float* weights,
                                              uint16_t* grad_rows, float* grad_weights, int T,
                                              int K, int L, lt_stream stream);

/*
 * Products of expert-sorted rows with 4-bit weights: for row r of expert e,
 *   out[r,m] = sum_c x[r,c] * (q[e,m,c] - 8) * scales[e,m,c/G]
 * with q[e,m,c] the 4-bit value in byte packed[e,m,c/2] (low four bits: even c),
 * products and sums in FP32, rounded once to bf16. Meant for the few rows of
 * decode steps, where reading the weights bounds the call: a matrix is read once
 * for 8 of its rows (16 where experts have many), again (mostly from L2) for more.
 * From about 32 rows per expert on a bf16 product with unpacked weights is faster
 * (256 experts of 2048 x 2048, G = 32: 143 us at 8 rows each, 351 at 32, 2305 at
 * 256; a batched bf16 product 364 at 64 and 424 at 256).
 * The order of a sum, and with it the last bits of a row, depends on N, E, M, C and G,
 * with one matrix on M, C and G alone.
 *   x [N, C] bf16, packed [E, M, C/2] bytes, scales [E, M, C/G] bf16,
 *   offsets [E+1] int32 (rows of expert e: offsets[e] .. offsets[e+1]-1, as
 *   latent_tail_dispatch writes it, or the part of it for some of the experts) or
 *   NULL with E == 1 (every row); out [N, M] bf16, every row of which is written.
 * Offsets are cut to [0, N] and to their running maximum, so that ones that run
 * backwards give empty experts. Rows that no expert owns, before offsets[0] and
 * from offsets[E] on, give zeros.
 * Limits: 0 <= N <= 2^24, 1 <= E <= 1024, 8 <= M <= 1048576 with M % 8 == 0,
 * G = 32, 64 or 128, C a multiple of G and at most 16384.
 */
LT_API lt_status latent_tail_expert_matvec4(const uint16_t* x, const uint8_t* packed,
                                            const uint16_t* scales, const int32_t* offsets,
                                            uint16_t* out, int N, int E, int M, int C, int G,
                                            lt_stream stream);

/*
 * Diagnostic as latent_tail_selftest_wait_timeout, for the waits of
 * latent_tail_expert_matvec4: the same call with waits of limit_us microseconds
 * (1 .. 1000000), in which tiles from copied_tiles (>= 0) on are never copied to the
 * SMs. Their waits expire; latent_tail_check reports LT_ERR_TIMEOUT. Elements of out
 * are then either the call's result or untouched.
 */
LT_API lt_status latent_tail_selftest_expert_matvec4_timeout(
    const uint16_t* x, const uint8_t* packed, const uint16_t* scales, const int32_t* offsets,
    uint16_t* out, int N, int E, int M, int C, int G, int copied_tiles, unsigned int limit_us,
    lt_stream stream);

/* What the gate of latent_tail_residual_norm holds. */
typedef enum lt_gate {
  LT_GATE_NONE = 0,    /* no gate (gate == NULL): 1                */
  LT_GATE_TOKEN = 1,   /* gate [T] fp32, one factor per token      */
  LT_GATE_CHANNEL = 2, /* gate [H] fp32, one factor per channel    */
  LT_GATE_FULL = 3     /* gate [T, H] bf16, one factor per element */
} lt_gate;

/* Type of the residual stream (residual, residual_out and their gradients). */
typedef enum lt_residual {
  LT_RESIDUAL_BF16 = 0,
  LT_RESIDUAL_FP32 = 1
} lt_residual;

/*
 * The norm after a block, its gate, the scaled residual sum and the norm before
 * the next block in one pass, in FP32:
 *   u[t,h]            = block[t,h] * rsqrt(mean_h block[t,h]^2 + eps) * post_weight[h]
 *                       (block[t,h] itself when post_weight is NULL)
 *   v[t,h]            = residual_scale * residual[t,h] + gate * u[t,h]
 *   residual_out[t,h] = v rounded to the residual's type
 *   next_out[t,h]     = bf16_rn(v[t,h] * rsqrt(mean_h v[t,h]^2 + eps) * next_weight[h])
 *                       (not computed when next_weight and next_out are NULL; the
 *                       norm takes v before its rounding)
 *   block [T, H] bf16 (e.g. the tail's out), residual [T, H], post_weight and
 *   next_weight [H] fp32 or NULL; residual_out may be exactly residual (in place).
 * Limits: 8 <= H <= 16384, H % 8 == 0, 0 <= T <= 2^24; residual_scale finite.
 */
LT_API lt_status latent_tail_residual_norm(const uint16_t* block, const void* residual,
                                           const float* post_weight, const void* gate,
                                           const float* next_weight, void* residual_out,
                                           uint16_t* next_out, int T, int H,
                                           lt_gate gate_kind, lt_residual residual_type,
                                           float residual_scale, float eps, lt_stream stream);

/*
 * Bytes of device workspace latent_tail_residual_norm_backward needs: the partial
 * sums of the gradients that add up over tokens (post_weight, next_weight, a
 * channel gate). The size covers every choice of optional arguments. Returns 0
 * for T <= 0 or invalid shapes. Host-only.
 */
LT_API size_t latent_tail_residual_norm_backward_workspace_size(int T, int H);

/*
 * Gradient of latent_tail_residual_norm at its inputs, from the gradients of its
 * outputs and the stored residual_out (which stands for v):
 *   grad_residual_out [T, H] (residual's type) or NULL (zero), grad_next [T, H]
 *   bf16 (given exactly when next_weight is; at least one of the two), block,
 *   residual_out, post_weight, gate and next_weight as in the forward call;
 *   grad_block [T, H] bf16, grad_residual [T, H] (residual's type),
 *   grad_post_weight, grad_next_weight [H] fp32 (given exactly when the weight is),
 *   grad_gate (shape and type of the gate; given exactly when the gate is).
 * With T == 0 the gradients of the weights and of a channel gate are zeros.
 */
LT_API lt_status latent_tail_residual_norm_backward(
    const void* grad_residual_out, const uint16_t* grad_next, const uint16_t* block,
    const void* residual_out, const float* post_weight, const void* gate,
    const float* next_weight, uint16_t* grad_block, void* grad_residual,
    float* grad_post_weight, void* grad_gate, float* grad_next_weight, int T, int H,
    lt_gate gate_kind, lt_residual residual_type, float residual_scale, float eps,
    void* workspace, size_t workspace_bytes, lt_stream stream);

/*
 * Diagnostics as latent_tail_selftest_expert_matvec4_timeout, for the waits of
 * latent_tail_residual_norm and its gradient: token rows from copied_rows (an even
 * number >= 0) on are never copied to the SMs. Shapes whose kernel loads its rows
 * directly (the forward call with fewer tokens than SMs and H <= 8192, or H < 520; the
 * gradient with H <= 512) have no such waits and give the whole result. Elements of the
 * outputs with a token index, an in-place residual among them, are then either the
 * call's result or untouched; the sums over tokens are incomplete.
 */
LT_API lt_status latent_tail_selftest_residual_norm_timeout(
    const uint16_t* block, const void* residual, const float* post_weight, const void* gate,
    const float* next_weight, void* residual_out, uint16_t* next_out, int T, int H,
    lt_gate gate_kind, lt_residual residual_type, float residual_scale, float eps,
    int copied_rows, unsigned int limit_us, lt_stream stream);

LT_API lt_status latent_tail_selftest_residual_norm_backward_timeout(
    const void* grad_residual_out, const uint16_t* grad_next, const uint16_t* block,
    const void* residual_out, const float* post_weight, const void* gate,
    const float* next_weight, uint16_t* grad_block, void* grad_residual,
    float* grad_post_weight, void* grad_gate, float* grad_next_weight, int T, int H,
    lt_gate gate_kind, lt_residual residual_type, float residual_scale, float eps,
    void* workspace, size_t workspace_bytes, int copied_rows, unsigned int limit_us,
    lt_stream stream);

/*
 * ---------------------------------------------------------------------------
 * The experts in bf16, for prefill and training, with their gradients. Rows are
 * sorted by expert as latent_tail_dispatch writes them:
 *
 *   latent_tail_dispatch -> latent_tail_expert_gated -> latent_tail_expert_matmul
 *     -> latent_tail_combine
 *
 * and with one matrix (E == 1, offsets NULL) the same calls are a dense block, such
 * as the shared expert. In all of them
 *   offsets [E+1] int32 (rows of expert e: offsets[e] .. offsets[e+1]-1) or NULL with
 *   E == 1 (every row). Offsets are cut to [0, N] and to their running maximum; rows
 *   that no expert owns give zeros, and experts without rows zero gradients. For some
 *   of the experts of a dispatch offsets may point into its array, at a multiple of
 *   four experts (16-byte alignment, as for every pointer).
 * Sums are FP32 on the tensor cores, results are rounded once to bf16; the order of a
 * sum, and with it the last bits of a result, depends on the sizes (N, E, F or M, C),
 * on whether offsets are given and on the device, not on the offsets themselves nor on
 * what is kept.
 * Limits: 0 <= N <= 2^24, 1 <= E <= 1024, C, M and 2F multiples of 8 from 8 to 65536
 * (F a multiple of 8).
 * With N == 0 the gradients of weights are zeros.
 */

/* The activation a of a gated block. */
typedef enum lt_activation {
  LT_ACTIVATION_SILU = 0, /* g * sigmoid(g) */
  LT_ACTIVATION_GELU = 1  /* the tanh form: g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
} lt_activation;

/* How the projections of a gated block are kept for its backward pass. */
typedef enum lt_saved {
  LT_SAVED_NONE = 0, /* not kept */
  LT_SAVED_BF16 = 1, /* saved [N, 2, F] bf16: gate, then up, of each row */
  LT_SAVED_8BIT = 2  /* saved [N, 2, F] int8 with exponents [N, 2, ceil(F/16)], as
                        latent_tail_quantize8 writes them for 2N rows of F columns */
} lt_saved;

/*
 * Both projections of a gated feed-forward block, its activation and the product in one
 * kernel: for row r of expert e
 *   g = sum_c x[r,c] weights[e,f,c],  u = sum_c x[r,c] weights[e,F+f,c]
 *   hidden[r,f] = bf16_rn(a(g) * u)
 * and, where saved is given, g and u as saved_kind says (rounded from FP32).
 *   x [N, C] bf16, weights [E, 2F, C] bf16; hidden [N, F] bf16, saved and
 *   saved_exponents outputs by saved_kind (NULL where it has none).
 */
LT_API lt_status latent_tail_expert_gated(const uint16_t* x, const uint16_t* weights,
                                          const int32_t* offsets, uint16_t* hidden, void* saved,
                                          uint8_t* saved_exponents, int N, int E, int F, int C,
                                          lt_activation activation, lt_saved saved_kind,
                                          lt_stream stream);

/*
 * Diagnostic as latent_tail_selftest_expert_matmul_timeout (below), for the waits of
 * latent_tail_expert_gated: each element of hidden and of what is kept is the call's result
 * or untouched.
 */
LT_API lt_status latent_tail_selftest_expert_gated_timeout(
    const uint16_t* x, const uint16_t* weights, const int32_t* offsets, uint16_t* hidden,
    void* saved, uint8_t* saved_exponents, int N, int E, int F, int C, lt_activation activation,
    lt_saved saved_kind, int copied_tiles, unsigned int limit_us, lt_stream stream);

/*
 * Bytes of device workspace latent_tail_expert_gated_backward needs: the gradient at both
 * projections, [N, 2F] bf16. Returns 0 for N <= 0 or invalid shapes. Host-only.
 */
LT_API size_t latent_tail_expert_gated_backward_workspace_size(int N, int F);

/*
 * Gradient of latent_tail_expert_gated, from the projections g and u that it kept
 * (saved_kind bf16 or 8 bits):
 *   dg = grad_hidden * u * a'(g), du = grad_hidden * a(g)   (rounded to bf16: operands
 *                                                             of the tensor cores)
 *   grad_x[r,c]          = sum_f dg[r,f] weights[e,f,c] + du[r,f] weights[e,F+f,c]
 *   grad_weights[e,f,c]  = sum over e's rows of dg[r,f] x[r,c], likewise F+f with du
 *   hidden[r,f]          = bf16_rn(a(g) * u) once more, for the gradient of the product
 *                          behind the block
 *   Each output may be NULL (not wanted), not all three; weights is read for grad_x
 *   alone, x for grad_weights alone, grad_hidden and the workspace for these two, and
 *   each may be NULL where it is not read.
 */
LT_API lt_status latent_tail_expert_gated_backward(
    const uint16_t* grad_hidden, const uint16_t* x, const uint16_t* weights, const void* saved,
    const uint8_t* saved_exponents, const int32_t* offsets, uint16_t* grad_x,
    uint16_t* grad_weights, uint16_t* hidden, int N, int E, int F, int C,
    lt_activation activation, lt_saved saved_kind, void* workspace, size_t workspace_bytes,
    lt_stream stream);

/*
 * Products of expert-sorted rows with bf16 weights: out[r,m] = sum_c x[r,c] weights[e,m,c]
 * for row r of expert e.
 *   x [N, C], weights [E, M, C], out [N, M], all bf16.
 */
LT_API lt_status latent_tail_expert_matmul(const uint16_t* x, const uint16_t* weights,
                                           const int32_t* offsets, uint16_t* out, int N, int E,
                                           int M, int C, lt_stream stream);

/*
 * Diagnostic as latent_tail_selftest_expert_matvec4_timeout, for the waits of
 * latent_tail_expert_matmul: tiles from copied_tiles (>= 0) on, in the order in which the
 * kernel takes them, are never copied to the SMs. Calls of few rows (up to 64, by the size
 * of the weights) load their operands directly, have no such waits and give the whole
 * result.
 */
LT_API lt_status latent_tail_selftest_expert_matmul_timeout(
    const uint16_t* x, const uint16_t* weights, const int32_t* offsets, uint16_t* out, int N,
    int E, int M, int C, int copied_tiles, unsigned int limit_us, lt_stream stream);

/*
 * Gradient of latent_tail_expert_matmul:
 *   grad_x[r,c]         = sum_m grad_out[r,m] weights[e,m,c]
 *   grad_weights[e,m,c] = sum over e's rows of grad_out[r,m] x[r,c]
 *   Each output may be NULL (not wanted), not both; weights is read for grad_x alone, x
 *   for grad_weights alone, and each may be NULL where it is not read.
 */
LT_API lt_status latent_tail_expert_matmul_backward(const uint16_t* grad_out, const uint16_t* x,
                                                    const uint16_t* weights,
                                                    const int32_t* offsets, uint16_t* grad_x,
                                                    uint16_t* grad_weights, int N, int E, int M,
                                                    int C, lt_stream stream);

/*
 * Diagnostic as latent_tail_selftest_expert_matmul_timeout, for the waits of
 * latent_tail_expert_matmul_backward (of the kernel of each gradient): each element of a
 * gradient is the call's result or untouched.
 */
LT_API lt_status latent_tail_selftest_expert_matmul_backward_timeout(
    const uint16_t* grad_out, const uint16_t* x, const uint16_t* weights, const int32_t* offsets,
    uint16_t* grad_x, uint16_t* grad_weights, int N, int E, int M, int C, int copied_tiles,
    unsigned int limit_us, lt_stream stream);

/*
 * Activations in 8 bits: per row and 16 columns (fewer behind the last multiple of 16) a
 * power of two 2^(e-127), e >= 1 the least for which the largest magnitude rounds to at
 * most 127 of it, and the values' integers:
 *   values[t,c]    = round(x[t,c] / 2^(e-127))      (to nearest even)
 *   exponents[t,g] = e, 0 for a group of zeros, 255 for one that holds an infinity or a
 *                    NaN (its values are 0)
 * so that a value is off by at most 1/127 of its group's largest magnitude (half a unit;
 * the largest magnitude is at least 63.5 units). Groups below 2^-126 * 63.5 round to that
 * power of two. (Where the values are FP32, as in latent_tail_expert_gated, magnitudes
 * below 2^-133 count as zeros.) At the other end, in a group whose largest magnitude is at
 * least 127.5 * 2^121 (of bf16 values its largest alone, 255/128 * 2^127), magnitudes from
 * 63.5 * 2^122 on (that one and the one below) round to 64 * 2^122 = 2^128, which reads back
 * as an infinity.
 *   x [T, C] bf16; values [T, C], exponents [T, ceil(C/16)].
 * Limits: 0 <= T <= 2^24, C a multiple of 8 from 8 to 65536.
 */
LT_API lt_status latent_tail_quantize8(const uint16_t* x, int8_t* values, uint8_t* exponents,
                                       int T, int C, lt_stream stream);

/*
 * out[t,c] = values[t,c] * 2^(exponents[t,g]-127) in bf16, which holds it exactly (values
 * of -128, which latent_tail_quantize8 does not write, too); zeros for exponent 0 and NaNs
 * for 255. Products past bf16's range give infinities (latent_tail_quantize8 writes them
 * for the largest magnitudes alone, as above).
 */
LT_API lt_status latent_tail_dequantize8(const int8_t* values, const uint8_t* exponents,
                                         uint16_t* out, int T, int C, lt_stream stream);

/* Static, human-readable name of a status code. Never NULL. */
LT_API const char* latent_tail_status_string(lt_status status);

#ifdef __cplusplus
}
#endif

#endif /* LATENT_TAIL_H */
