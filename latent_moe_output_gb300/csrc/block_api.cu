// C ABI of the operators around the tail (declared in include/latent_tail.h):
// host-side argument validation and the launches.
#include "block_launch.h"
#include "host_checks.h"

#include <cmath>
#include <vector>

using namespace lt;

namespace {

lt_status check_choices(int T, int K) {
  if (T < 0 || T > (1 << 24) || K < 1 || K > kMaxChoices) return LT_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * K > kMaxSlots) return LT_ERR_INVALID_ARG;
  return LT_OK;
}

lt_status check_width(int L, int most) {
  if (L < 8 || L > most) return LT_ERR_INVALID_ARG;
  return L % 8 != 0 ? LT_ERR_ALIGNMENT : LT_OK;
}

// No output may overlap an input or another output; null spans are skipped.
// `in_place`: an output may be exactly an input that begins here (same range).
bool disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins,
              const void* in_place = nullptr) {
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    if (a->lo == 0) continue;
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (b->lo != 0 && overlaps(*a, *b)) return false;
    for (const Span& in : ins) {
      if (in.lo == 0 || !overlaps(*a, in)) continue;
      if (in_place != nullptr && a->lo == in.lo && a->hi == in.hi &&
          in.lo == reinterpret_cast<uintptr_t>(in_place))
        continue;
      return false;
    }
  }
  return true;
}

// Alignment of optional pointers (null is fine).
lt_status check_optional(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return LT_ERR_ALIGNMENT;
  return LT_OK;
}

size_t gate_bytes(int kind, int T, int H) {
  switch (kind) {
    case LT_GATE_TOKEN: return static_cast<size_t>(T) * 4;
    case LT_GATE_CHANNEL: return static_cast<size_t>(H) * 4;
    case LT_GATE_FULL: return static_cast<size_t>(T) * H * 2;
    default: return 0;
  }
}

lt_status check_norm(int T, int H, int gate_kind, const void* gate, int residual_type,
                     float scale, float eps) {
  if (T < 0 || T > (1 << 24)) return LT_ERR_INVALID_ARG;
  const lt_status st = check_width(H, 16384);
  if (st != LT_OK) return st;
  if (gate_kind < LT_GATE_NONE || gate_kind > LT_GATE_FULL) return LT_ERR_INVALID_ARG;
  if (residual_type != LT_RESIDUAL_BF16 && residual_type != LT_RESIDUAL_FP32)
    return LT_ERR_INVALID_ARG;
  if (gate_kind == LT_GATE_NONE && gate != nullptr) return LT_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(eps) || !(eps > 0.f)) return LT_ERR_INVALID_ARG;
  return LT_OK;
}

lt_status zero(void* p, size_t bytes, cudaStream_t s) {
  return p == nullptr ? LT_OK : launch_status(cudaMemsetAsync(p, 0, bytes, s));
}

// Limits of a self-test of expired waits.
bool test_limits(int copied, unsigned int limit_us, RingLimits* ring) {
  if (copied < 0 || limit_us < 1 || limit_us > 1000000) return false;
  *ring = RingLimits{copied, static_cast<uint64_t>(limit_us) * 1000u};
  return true;
}

lt_status expert_matvec4(const uint16_t* x, const uint8_t* packed, const uint16_t* scales,
                         const int32_t* offsets, uint16_t* out, int N, int E, int M, int C, int G,
                         const RingLimits& ring, lt_stream stream) {
  if (N < 0 || N > (1 << 24) || E < 1 || E > kMaxExperts || M < 8 || M > (1 << 20))
    return LT_ERR_INVALID_ARG;
  if (G != 32 && G != 64 && G != 128) return LT_ERR_INVALID_ARG;
  if (C < G || C > 16384) return LT_ERR_INVALID_ARG;
  if (M % 8 != 0 || C % G != 0) return LT_ERR_ALIGNMENT;
  if (offsets == nullptr && E != 1) return LT_ERR_INVALID_ARG;
  if (N == 0) return LT_OK;
  lt_status st = check_ptrs({x, packed, scales, out});
  if (st != LT_OK) return st;
  if ((st = check_optional({offsets})) != LT_OK) return st;
  const size_t em = static_cast<size_t>(E) * M;
  if (!disjoint({span(out, static_cast<size_t>(N) * M * 2)},
                {span(x, static_cast<size_t>(N) * C * 2), span(packed, em * (C / 2)),
                 span(scales, em * (C / G) * 2), span(offsets, static_cast<size_t>(E + 1) * 4)}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kMatvec4)) != LT_OK) return st;
  const Matvec4Args a{x, packed, scales, offsets, out, N, E, M, C, G, ring};
  return launch_status(launch_matvec4(a, *dev, reinterpret_cast<cudaStream_t>(stream)));
}

lt_status residual_norm(const uint16_t* block, const void* residual, const float* post_weight,
                        const void* gate, const float* next_weight, void* residual_out,
                        uint16_t* next_out, int T, int H, lt_gate gate_kind,
                        lt_residual residual_type, float residual_scale, float eps,
                        const RingLimits& ring, lt_stream stream) {
  lt_status st = check_norm(T, H, gate_kind, gate, residual_type, residual_scale, eps);
  if (st != LT_OK) return st;
  if (T == 0) return LT_OK;
  if ((next_weight == nullptr) != (next_out == nullptr)) return LT_ERR_INVALID_ARG;
  if ((st = check_ptrs({block, residual, residual_out})) != LT_OK) return st;
  if (gate_kind != LT_GATE_NONE && (st = check_ptrs({gate})) != LT_OK) return st;
  if ((st = check_optional({post_weight, next_weight, next_out})) != LT_OK) return st;
  const size_t th = static_cast<size_t>(T) * H;
  const size_t r_bytes = th * (residual_type == LT_RESIDUAL_FP32 ? 4 : 2);
  const size_t h_bytes = static_cast<size_t>(H) * 4;
  // In place: every element of block, residual and a full gate is read before the element
  // of residual_out that it enters is written. The vectors are read for each row.
  const Span gate_span = span(gate, gate_bytes(gate_kind, T, H));
  const bool full = gate_kind == LT_GATE_FULL;
  const auto outs = {span(residual_out, r_bytes), span(next_out, th * 2)};
  if (!disjoint(outs, {span(block, th * 2), span(residual, r_bytes), full ? gate_span : Span{0, 0}},
                residual) ||
      !disjoint(outs, {span(post_weight, h_bytes), full ? Span{0, 0} : gate_span,
                       span(next_weight, h_bytes)}))
    return LT_ERR_INVALID_ARG;
  // (residual_out == residual is the only in-place form: next_out has its own range)
  if (next_out != nullptr && static_cast<const void*>(next_out) == residual)
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kResidualNorm)) != LT_OK) return st;
  const ResidualNormArgs a{block, residual, post_weight, gate, next_weight, residual_out,
                           next_out, T, H, gate_kind, residual_type == LT_RESIDUAL_FP32,
                           residual_scale, eps, ring};
  return launch_status(launch_residual_norm(a, *dev, reinterpret_cast<cudaStream_t>(stream)));
}

size_t backward_workspace(int T, int H) {
  if (T <= 0 || T > (1 << 24) || check_width(H, 16384) != LT_OK) return 0;
  return round256(2 * static_cast<size_t>(residual_norm_partial_rows(T, H)) * H * sizeof(float));
}

lt_status residual_norm_backward(
    const void* grad_residual_out, const uint16_t* grad_next, const uint16_t* block,
    const void* residual_out, const float* post_weight, const void* gate,
    const float* next_weight, uint16_t* grad_block, void* grad_residual, float* grad_post_weight,
    void* grad_gate, float* grad_next_weight, int T, int H, lt_gate gate_kind,
    lt_residual residual_type, float residual_scale, float eps, void* workspace,
    size_t workspace_bytes, const RingLimits& ring, lt_stream stream) {
  lt_status st = check_norm(T, H, gate_kind, gate, residual_type, residual_scale, eps);
  if (st != LT_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t h_bytes = static_cast<size_t>(H) * 4;
  const lt::DeviceInfo* dev = nullptr;
  if (T == 0) {
    if ((st = check_optional({grad_post_weight, grad_next_weight, grad_gate})) != LT_OK) return st;
    if ((st = current_device(&dev, Operator::kResidualNorm)) != LT_OK) return st;
    if ((st = zero(grad_post_weight, h_bytes, s)) != LT_OK) return st;
    if ((st = zero(grad_next_weight, h_bytes, s)) != LT_OK) return st;
    return gate_kind == LT_GATE_CHANNEL ? zero(grad_gate, h_bytes, s) : LT_OK;
  }
  if ((post_weight == nullptr) != (grad_post_weight == nullptr) ||
      (next_weight == nullptr) != (grad_next_weight == nullptr) ||
      (next_weight == nullptr) != (grad_next == nullptr) ||
      (gate_kind == LT_GATE_NONE) != (grad_gate == nullptr) ||
      (grad_residual_out == nullptr && grad_next == nullptr))
    return LT_ERR_INVALID_ARG;
  if ((st = check_ptrs({block, residual_out, grad_block, grad_residual})) != LT_OK) return st;
  if (gate_kind != LT_GATE_NONE && (st = check_ptrs({gate})) != LT_OK) return st;
  if ((st = check_optional({grad_residual_out, grad_next, post_weight, next_weight,
                            grad_post_weight, grad_gate, grad_next_weight})) != LT_OK)
    return st;
  const size_t need = backward_workspace(T, H);
  if (workspace == nullptr || workspace_bytes < need) return LT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return LT_ERR_ALIGNMENT;
  const size_t th = static_cast<size_t>(T) * H;
  const size_t r_bytes = th * (residual_type == LT_RESIDUAL_FP32 ? 4 : 2);
  const size_t g_bytes = gate_bytes(gate_kind, T, H);
  if (!disjoint({span(grad_block, th * 2), span(grad_residual, r_bytes),
                 span(grad_post_weight, h_bytes), span(grad_gate, g_bytes),
                 span(grad_next_weight, h_bytes), span(workspace, need)},
                {span(grad_residual_out, r_bytes), span(grad_next, th * 2), span(block, th * 2),
                 span(residual_out, r_bytes), span(post_weight, h_bytes), span(gate, g_bytes),
                 span(next_weight, h_bytes)}))
    return LT_ERR_INVALID_ARG;
  if ((st = current_device(&dev, Operator::kResidualNorm)) != LT_OK) return st;
  const ResidualNormBackwardArgs a{
      grad_residual_out, grad_next, block, residual_out, post_weight, gate, next_weight,
      grad_block, grad_residual, grad_post_weight, grad_gate, grad_next_weight, T, H, gate_kind,
      residual_type == LT_RESIDUAL_FP32, residual_scale, eps, static_cast<float*>(workspace), ring};
  return launch_status(launch_residual_norm_backward(a, *dev, s));
}

}  // namespace

extern "C" {

LT_API size_t latent_tail_dispatch_workspace_size(int T, int K, int E) {
  if (T <= 0 || check_choices(T, K) != LT_OK || E < 1 || E > kMaxExperts) return 0;
  if (static_cast<int64_t>(T) * K <= kDispatchOneLaunch) return 0;
  return round256(static_cast<size_t>(kDispatchMaxChunks) * dispatch_counts_stride(E) *
                  sizeof(uint16_t));
}

LT_API lt_status latent_tail_dispatch(const uint16_t* x, const int32_t* expert_ids,
                                      uint16_t* rows, int32_t* offsets, int32_t* order,
                                      int32_t* position, int T, int K, int E, int L,
                                      void* workspace, size_t workspace_bytes, lt_stream stream) {
  lt_status st = check_choices(T, K);
  if (st != LT_OK) return st;
  if (E < 1 || E > kMaxExperts) return LT_ERR_INVALID_ARG;
  const bool copy = x != nullptr || rows != nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if ((st = check_ptrs({offsets})) != LT_OK) return st;
    const lt::DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev, Operator::kDispatch)) != LT_OK) return st;
    return zero(offsets, static_cast<size_t>(E + 1) * 4, s);
  }
  if (copy && (st = check_width(L, 16384)) != LT_OK) return st;
  if ((st = check_ptrs({expert_ids, offsets, order, position})) != LT_OK) return st;
  if (copy && (st = check_ptrs({x, rows})) != LT_OK) return st;
  const size_t need = latent_tail_dispatch_workspace_size(T, K, E);
  if (need != 0) {
    if (workspace == nullptr || workspace_bytes < need) return LT_ERR_WORKSPACE;
    if (!aligned16(workspace)) return LT_ERR_ALIGNMENT;
  }
  const size_t n = static_cast<size_t>(T) * K;
  if (!disjoint({span(rows, copy ? n * L * 2 : 0), span(offsets, static_cast<size_t>(E + 1) * 4),
                 span(order, n * 4), span(position, n * 4), span(need ? workspace : nullptr, need)},
                {span(x, copy ? static_cast<size_t>(T) * L * 2 : 0), span(expert_ids, n * 4)}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kDispatch)) != LT_OK) return st;
  const DispatchArgs a{x, expert_ids, rows, offsets, order, position, T, K, E, L,
                       static_cast<uint16_t*>(workspace)};
  return launch_status(launch_dispatch(a, *dev, s));
}

LT_API lt_status latent_tail_combine(const uint16_t* rows, const int32_t* position,
                                     const float* weights, uint16_t* out, int T, int K, int L,
                                     lt_stream stream) {
  lt_status st = check_choices(T, K);
  if (st != LT_OK) return st;
  if ((st = check_width(L, 16384)) != LT_OK) return st;
  if (T == 0) return LT_OK;
  if ((st = check_ptrs({rows, position, out})) != LT_OK) return st;
  if ((st = check_optional({weights})) != LT_OK) return st;
  const size_t n = static_cast<size_t>(T) * K;
  if (!disjoint({span(out, static_cast<size_t>(T) * L * 2)},
                {span(rows, n * L * 2), span(position, n * 4), span(weights, n * 4)}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != LT_OK) return st;
  const CombineArgs a{rows, position, weights, out, T, K, L};
  return launch_status(launch_combine(a, *dev, reinterpret_cast<cudaStream_t>(stream)));
}

LT_API lt_status latent_tail_combine_backward(const uint16_t* grad_out, const uint16_t* rows,
                                              const int32_t* position, const float* weights,
                                              uint16_t* grad_rows, float* grad_weights, int T,
                                              int K, int L, lt_stream stream) {
  lt_status st = check_choices(T, K);
  if (st != LT_OK) return st;
  if ((st = check_width(L, 16384)) != LT_OK) return st;
  if (T == 0) return LT_OK;
  if ((st = check_ptrs({grad_out, position, grad_rows})) != LT_OK) return st;
  if (grad_weights != nullptr && rows == nullptr) return LT_ERR_INVALID_ARG;
  if ((st = check_optional({rows, weights, grad_weights})) != LT_OK) return st;
  const size_t n = static_cast<size_t>(T) * K;
  if (!disjoint({span(grad_rows, n * L * 2), span(grad_weights, n * 4)},
                {span(grad_out, static_cast<size_t>(T) * L * 2), span(rows, n * L * 2),
                 span(position, n * 4), span(weights, n * 4)}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != LT_OK) return st;
  const CombineBackwardArgs a{grad_out, rows, position, weights, grad_rows, grad_weights, T, K, L};
  return launch_status(launch_combine_backward(a, *dev, reinterpret_cast<cudaStream_t>(stream)));
}

LT_API lt_status latent_tail_expert_matvec4(const uint16_t* x, const uint8_t* packed,
                                            const uint16_t* scales, const int32_t* offsets,
                                            uint16_t* out, int N, int E, int M, int C, int G,
                                            lt_stream stream) {
  return expert_matvec4(x, packed, scales, offsets, out, N, E, M, C, G, RingLimits{}, stream);
}

LT_API lt_status latent_tail_selftest_expert_matvec4_timeout(
    const uint16_t* x, const uint8_t* packed, const uint16_t* scales, const int32_t* offsets,
    uint16_t* out, int N, int E, int M, int C, int G, int copied_tiles, unsigned int limit_us,
    lt_stream stream) {
  RingLimits ring;
  if (!test_limits(copied_tiles, limit_us, &ring)) return LT_ERR_INVALID_ARG;
  return expert_matvec4(x, packed, scales, offsets, out, N, E, M, C, G, ring, stream);
}

LT_API lt_status latent_tail_residual_norm(const uint16_t* block, const void* residual,
                                           const float* post_weight, const void* gate,
                                           const float* next_weight, void* residual_out,
                                           uint16_t* next_out, int T, int H, lt_gate gate_kind,
                                           lt_residual residual_type, float residual_scale,
                                           float eps, lt_stream stream) {
  return residual_norm(block, residual, post_weight, gate, next_weight, residual_out, next_out, T,
                       H, gate_kind, residual_type, residual_scale, eps, RingLimits{}, stream);
}

LT_API lt_status latent_tail_selftest_residual_norm_timeout(
    const uint16_t* block, const void* residual, const float* post_weight, const void* gate,
    const float* next_weight, void* residual_out, uint16_t* next_out, int T, int H,
    lt_gate gate_kind, lt_residual residual_type, float residual_scale, float eps,
    int copied_rows, unsigned int limit_us, lt_stream stream) {
  RingLimits ring;
  if (!test_limits(copied_rows, limit_us, &ring)) return LT_ERR_INVALID_ARG;
  return residual_norm(block, residual, post_weight, gate, next_weight, residual_out, next_out, T,
                       H, gate_kind, residual_type, residual_scale, eps, ring, stream);
}

LT_API size_t latent_tail_residual_norm_backward_workspace_size(int T, int H) {
  return backward_workspace(T, H);
}

LT_API lt_status latent_tail_residual_norm_backward(
    const void* grad_residual_out, const uint16_t* grad_next, const uint16_t* block,
    const void* residual_out, const float* post_weight, const void* gate,
    const float* next_weight, uint16_t* grad_block, void* grad_residual, float* grad_post_weight,
    void* grad_gate, float* grad_next_weight, int T, int H, lt_gate gate_kind,
    lt_residual residual_type, float residual_scale, float eps, void* workspace,
    size_t workspace_bytes, lt_stream stream) {
  return residual_norm_backward(grad_residual_out, grad_next, block, residual_out, post_weight,
                                gate, next_weight, grad_block, grad_residual, grad_post_weight,
                                grad_gate, grad_next_weight, T, H, gate_kind, residual_type,
                                residual_scale, eps, workspace, workspace_bytes, RingLimits{},
                                stream);
}

LT_API lt_status latent_tail_selftest_residual_norm_backward_timeout(
    const void* grad_residual_out, const uint16_t* grad_next, const uint16_t* block,
    const void* residual_out, const float* post_weight, const void* gate,
    const float* next_weight, uint16_t* grad_block, void* grad_residual, float* grad_post_weight,
    void* grad_gate, float* grad_next_weight, int T, int H, lt_gate gate_kind,
    lt_residual residual_type, float residual_scale, float eps, void* workspace,
    size_t workspace_bytes, int copied_rows, unsigned int limit_us, lt_stream stream) {
  RingLimits ring;
  if (!test_limits(copied_rows, limit_us, &ring)) return LT_ERR_INVALID_ARG;
  return residual_norm_backward(grad_residual_out, grad_next, block, residual_out, post_weight,
                                gate, next_weight, grad_block, grad_residual, grad_post_weight,
                                grad_gate, grad_next_weight, T, H, gate_kind, residual_type,
                                residual_scale, eps, workspace, workspace_bytes, ring,
                                stream);
}

}  // extern "C"
