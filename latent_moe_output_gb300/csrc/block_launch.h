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

cudaError_t setup_dispatch(const DeviceInfo& dev);
cudaError_t setup_matvec4(const DeviceInfo& dev);
cudaError_t setup_residual_norm(const DeviceInfo& dev);

}  // namespace lt
