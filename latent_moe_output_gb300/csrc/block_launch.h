// Library-internal host interface between the C-ABI layer (block_api.cu) and
// the kernels of the operators around the tail. Not installed, not part of the ABI.
#pragma once

#include "launch.h"

namespace lt {

constexpr int kMaxChoices = 64;            // K
constexpr int kMaxExperts = 1024;          // E
constexpr int kMaxSlots = 1 << 24;         // T * K

struct DispatchArgs {
  const uint16_t* x;    // [T,L] or null (sort alone)
  const int32_t* ids;   // [T,K]
  uint16_t* rows;       // [T*K,L] or null
  int32_t* offsets;     // [E+1]
  int32_t* order;       // [T*K]
  int32_t* position;    // [T,K]
  int T, K, E, L;
  uint16_t* counts;     // workspace: [chunks][counts_stride(E)]
};

// Up to this many choices one kernel sorts and copies (see dispatch.cu).
constexpr int kDispatchOneLaunch = 2048;
// Most chunks the choices of a larger call are cut into.
constexpr int kDispatchMaxChunks = 304;
// Counts per chunk: one per expert and one for choices without an expert,
// padded to whole 16-byte vectors.
constexpr int dispatch_counts_stride(int E) { return (E + 1 + 7) / 8 * 8; }

struct CombineArgs {
  const uint16_t* rows;     // [T*K,L]
  const int32_t* position;  // [T,K]
  const float* weights;     // [T,K] or null
  uint16_t* out;            // [T,L]
  int T, K, L;
};

struct CombineBackwardArgs {
  const uint16_t* grad_out;  // [T,L]
  const uint16_t* rows;      // [T*K,L] or null (no grad_weights)
  const int32_t* position;   // [T,K]
  const float* weights;      // [T,K] or null
  uint16_t* grad_rows;       // [T*K,L]
  float* grad_weights;       // [T,K] or null
  int T, K, L;
};

// 2-D map of bytes, row-major [rows, bytes], with a (box_bytes x box_rows) box: 128
// bytes with 128-byte swizzle, else none. Returns false if the driver rejects it.
bool make_map_u8(CUtensorMap* map, const void* base, uint64_t rows, uint64_t bytes,
                 uint32_t box_bytes, uint32_t box_rows);

// 3-D map of a row-major bf16 [rows, cols] array, cols a multiple of 64, as
// (64 columns, rows, 64-column chunks): one box brings box_chunks chunks of box_rows
// rows, each chunk a 128-byte-swizzled block. Returns false if the driver rejects it.
bool make_map_bf16_rows64(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                          uint32_t box_rows, uint32_t box_chunks);

// Map of a bf16 array of `rank` dimensions (innermost first; strides in bytes from the
// second on) with 128-byte swizzle; box[0] is 64. Returns false if the driver rejects it.
bool make_map_bf16_nd(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box);

// Limits of a kernel's ring of copies: work (tiles, rows) from `copied` on is never
// copied in, and a wait runs out after limit_ns. Calls leave nothing out; the self-tests
// of expired waits do.
struct RingLimits {
  int64_t copied = INT64_MAX;
  uint64_t limit_ns = kWaitLimitNs;
};

struct Matvec4Args {
  const uint16_t* x;       // [N,C]
  const uint8_t* packed;   // [E,M,C/2]
  const uint16_t* scales;  // [E,M,C/G]
  const int32_t* offsets;  // [E+1] or null (E == 1)
  uint16_t* out;           // [N,M]
  int N, E, M, C, G;
  RingLimits ring;
};

enum GateKind { kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateFull = 3 };

struct ResidualNormArgs {
  const uint16_t* block;   // [T,H]
  const void* residual;    // [T,H]
  const float* post;       // [H] or null
  const void* gate;        // by gate_kind, or null
  const float* next;       // [H] or null
  void* residual_out;      // [T,H]
  uint16_t* next_out;      // [T,H] or null
  int T, H;
  int gate_kind;
  bool residual_f32;
  float scale, eps;
  RingLimits ring;
};

struct ResidualNormBackwardArgs {
  const void* grad_residual_out;  // [T,H] or null
  const uint16_t* grad_next;      // [T,H] or null
  const uint16_t* block;          // [T,H]
  const void* residual_out;       // [T,H]
  const float* post;              // [H] or null
  const void* gate;
  const float* next;              // [H] or null
  uint16_t* grad_block;           // [T,H]
  void* grad_residual;            // [T,H]
  float* grad_post;               // [H] or null
  void* grad_gate;
  float* grad_next_weight;        // [H] or null
  int T, H;
  int gate_kind;
  bool residual_f32;
  float scale, eps;
  float* partials;                // workspace: [2][rows][H]
  RingLimits ring;
};

enum Activation { kActSilu = 0, kActGelu = 1 };
enum SavedKind { kSavedNone = 0, kSavedBf16 = 1, kSaved8 = 2 };

struct ExpertGatedArgs {
  const uint16_t* x;        // [N,C]
  const uint16_t* weights;  // [E,2F,C], gate rows first
  const int32_t* offsets;   // [E+1] or null (E == 1)
  uint16_t* hidden;         // [N,F]
  void* saved;              // [N,2,F] bf16 or 8 bits, or null
  uint8_t* exponents;       // [N,2,ceil(F/16)] or null
  int N, E, F, C;
  int act, saved_kind;
  RingLimits ring;
};

// out = x times each expert's [M,K] weights (or [K,M] ones, transposed).
struct ExpertRowsArgs {
  const uint16_t* x;        // [N,K]
  const uint16_t* weights;  // [E,M,K]; transposed: [E,K,M]
  const int32_t* offsets;
  uint16_t* out;            // [N,M]
  int N, E, M, K;
  bool transposed;
  RingLimits ring;
};

// grad_weights[e] = grad^T x over the rows of expert e.
struct ExpertWeightsArgs {
  const uint16_t* grad;     // [N,M]
  const uint16_t* x;        // [N,C]
  const int32_t* offsets;
  uint16_t* grad_weights;   // [E,M,C]
  int N, E, M, C;
  RingLimits ring;
};

// Whether experts_few.cu takes a call of N rows of C columns with E matrices, whose result
// has M columns.
bool few_rows(const int32_t* offsets, int N, int E, int M, int C, bool gated,
              const DeviceInfo& dev);

// The gradient at both projections, and the product again, from what was kept of them.
struct GatedGradArgs {
  const uint16_t* grad_hidden;  // [N,F]
  const void* saved;            // [N,2,F]
  const uint8_t* exponents;     // [N,2,ceil(F/16)] or null
  const int32_t* offsets;
  uint16_t* grad_pre;           // [N,2F] or null (not wanted)
  uint16_t* hidden;             // [N,F] or null
  int N, E, F;
  int act, saved_kind;
};

struct Quantize8Args {
  const uint16_t* x;   // [T,C] (quantize8)
  int8_t* values;      // [T,C]
  uint8_t* exponents;  // [T,ceil(C/16)]
  uint16_t* out;       // [T,C] (dequantize8)
  int T, C;
};

// SMs that a workspace size computed without a device allows for.
constexpr int kMaxSms = 304;
// Rows of partial sums that a call of T tokens of width H may write (bounds the
// workspace without knowing the device).
int residual_norm_partial_rows(int T, int H);

cudaError_t launch_dispatch(const DispatchArgs& a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_combine(const CombineArgs& a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_combine_backward(const CombineBackwardArgs& a, const DeviceInfo& dev,
                                    cudaStream_t stream);
cudaError_t launch_matvec4(const Matvec4Args& a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_residual_norm(const ResidualNormArgs& a, const DeviceInfo& dev,
                                 cudaStream_t stream);
cudaError_t launch_residual_norm_backward(const ResidualNormBackwardArgs& a,
                                          const DeviceInfo& dev, cudaStream_t stream);

cudaError_t launch_expert_gated(const ExpertGatedArgs& a, const DeviceInfo& dev,
                                cudaStream_t stream);
cudaError_t launch_expert_rows(const ExpertRowsArgs& a, const DeviceInfo& dev,
                               cudaStream_t stream);
cudaError_t launch_expert_gated_few(const ExpertGatedArgs& a, cudaStream_t stream);
cudaError_t launch_expert_rows_few(const ExpertRowsArgs& a, cudaStream_t stream);
cudaError_t launch_expert_weights(const ExpertWeightsArgs& a, const DeviceInfo& dev,
                                  cudaStream_t stream);
cudaError_t launch_gated_grad(const GatedGradArgs& a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_quantize8(const Quantize8Args& a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_dequantize8(const Quantize8Args& a, const DeviceInfo& dev, cudaStream_t stream);

cudaError_t setup_dispatch(const DeviceInfo& dev);
cudaError_t setup_matvec4(const DeviceInfo& dev);
cudaError_t setup_residual_norm(const DeviceInfo& dev);
cudaError_t setup_experts(const DeviceInfo& dev);

}  // namespace lt
