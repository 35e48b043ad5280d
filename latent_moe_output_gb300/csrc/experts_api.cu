// C ABI of the bf16 experts and of activations in 8 bits (declared in
// include/latent_tail.h): host-side argument validation and the launches.
#include "block_launch.h"
#include "host_checks.h"

using namespace lt;

namespace {

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxWidth = 1 << 16;

lt_status check_width(int n) {
  if (n < 8 || n > kMaxWidth) return LT_ERR_INVALID_ARG;
  return n % 8 != 0 ? LT_ERR_ALIGNMENT : LT_OK;
}

// Sizes of products of N rows with E matrices of M x C.
lt_status check_sizes(int N, int E, int M, int C, const int32_t* offsets) {
  if (N < 0 || N > kMaxRows || E < 1 || E > kMaxExperts) return LT_ERR_INVALID_ARG;
  for (const int n : {M, C}) {
    const lt_status st = check_width(n);
    if (st != LT_OK) return st;
  }
  return offsets == nullptr && E != 1 ? LT_ERR_INVALID_ARG : LT_OK;
}

lt_status check_optional(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return LT_ERR_ALIGNMENT;
  return LT_OK;
}

size_t bytes_of(int64_t a, int64_t b, int64_t each) { return static_cast<size_t>(a * b * each); }
int64_t groups8(int C) { return (C + 15) / 16; }

bool known(int act) { return act == LT_ACTIVATION_SILU || act == LT_ACTIVATION_GELU; }

// Kept projections: their kind, and the arrays that it needs.
lt_status check_saved(int kind, const void* saved, const void* exponents) {
  if ((kind == LT_SAVED_NONE) != (saved == nullptr)) return LT_ERR_INVALID_ARG;
  if ((kind == LT_SAVED_8BIT) != (exponents != nullptr)) return LT_ERR_INVALID_ARG;
  return check_optional({saved, exponents});
}

size_t saved_bytes(int kind, int N, int F) {
  return bytes_of(N, 2 * static_cast<int64_t>(F), kind == LT_SAVED_BF16 ? 2 : 1);
}

// No output may overlap an input or another output; null spans are skipped.
bool disjoint(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    if (a->lo == 0) continue;
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (b->lo != 0 && overlaps(*a, *b)) return false;
    for (const Span& in : ins)
      if (in.lo != 0 && overlaps(*a, in)) return false;
  }
  return true;
}

cudaStream_t raw(lt_stream s) { return reinterpret_cast<cudaStream_t>(s); }

lt_status zero_weights(void* p, int E, int M, int C, lt_stream stream) {
  if (p == nullptr) return LT_OK;
  lt_status st = check_optional({p});
  if (st != LT_OK) return st;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != LT_OK) return st;
  return launch_status(cudaMemsetAsync(p, 0, static_cast<size_t>(E) * bytes_of(M, C, 2),
                                       raw(stream)));
}

lt_status expert_matmul(const uint16_t* x, const uint16_t* weights, const int32_t* offsets,
                        uint16_t* out, int N, int E, int M, int C, const RingLimits& ring,
                        lt_stream stream) {
  lt_status st = check_sizes(N, E, M, C, offsets);
  if (st != LT_OK || N == 0) return st;
  if ((st = check_ptrs({x, weights, out})) != LT_OK) return st;
  if ((st = check_optional({offsets})) != LT_OK) return st;
  if (!disjoint({span(out, bytes_of(N, M, 2))},
                {span(x, bytes_of(N, C, 2)), span(weights, E * bytes_of(M, C, 2)),
                 span(offsets, bytes_of(E + 1, 4, 1))}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kExperts)) != LT_OK) return st;
  const ExpertRowsArgs a{x, weights, offsets, out, N, E, M, C, false, ring};
  return launch_status(launch_expert_rows(a, *dev, raw(stream)));
}

lt_status expert_gated(const uint16_t* x, const uint16_t* weights, const int32_t* offsets,
                       uint16_t* hidden, void* saved, uint8_t* saved_exponents, int N, int E, int F,
                       int C, lt_activation activation, lt_saved saved_kind,
                       const RingLimits& ring, lt_stream stream) {
  lt_status st = check_sizes(N, E, F, C, offsets);
  if (st != LT_OK) return st;
  if (F > kMaxWidth / 2 || !known(activation)) return LT_ERR_INVALID_ARG;
  if (saved_kind != LT_SAVED_NONE && saved_kind != LT_SAVED_BF16 && saved_kind != LT_SAVED_8BIT)
    return LT_ERR_INVALID_ARG;
  if (N == 0) return LT_OK;
  if ((st = check_saved(saved_kind, saved, saved_exponents)) != LT_OK) return st;
  if ((st = check_ptrs({x, weights, hidden})) != LT_OK) return st;
  if ((st = check_optional({offsets})) != LT_OK) return st;
  if (!disjoint({span(hidden, bytes_of(N, F, 2)), span(saved, saved_bytes(saved_kind, N, F)),
                 span(saved_exponents, bytes_of(N, 2, groups8(F)))},
                {span(x, bytes_of(N, C, 2)), span(weights, E * bytes_of(2 * F, C, 2)),
                 span(offsets, bytes_of(E + 1, 4, 1))}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kExperts)) != LT_OK) return st;
  const ExpertGatedArgs a{x, weights, offsets, hidden, saved, saved_exponents, N, E, F, C,
                          activation, saved_kind, ring};
  return launch_status(launch_expert_gated(a, *dev, raw(stream)));
}

lt_status expert_matmul_backward(const uint16_t* grad_out, const uint16_t* x,
                                 const uint16_t* weights, const int32_t* offsets, uint16_t* grad_x,
                                 uint16_t* grad_weights, int N, int E, int M, int C,
                                 const RingLimits& ring, lt_stream stream) {
  lt_status st = check_sizes(N, E, M, C, offsets);
  if (st != LT_OK) return st;
  if (N == 0) return zero_weights(grad_weights, E, M, C, stream);
  if (grad_x == nullptr && grad_weights == nullptr) return LT_ERR_INVALID_ARG;
  if ((st = check_ptrs({grad_out})) != LT_OK) return st;
  if ((grad_x != nullptr && weights == nullptr) || (grad_weights != nullptr && x == nullptr))
    return LT_ERR_INVALID_ARG;
  if ((st = check_optional({x, weights, offsets, grad_x, grad_weights})) != LT_OK) return st;
  const size_t w_bytes = E * bytes_of(M, C, 2);
  if (!disjoint({span(grad_x, bytes_of(N, C, 2)), span(grad_weights, w_bytes)},
                {span(grad_out, bytes_of(N, M, 2)), span(x, bytes_of(N, C, 2)),
                 span(weights, w_bytes), span(offsets, bytes_of(E + 1, 4, 1))}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kExperts)) != LT_OK) return st;
  if (grad_x != nullptr) {
    const ExpertRowsArgs r{grad_out, weights, offsets, grad_x, N, E, C, M, true, ring};
    if ((st = launch_status(launch_expert_rows(r, *dev, raw(stream)))) != LT_OK) return st;
  }
  if (grad_weights != nullptr) {
    const ExpertWeightsArgs w{grad_out, x, offsets, grad_weights, N, E, M, C, ring};
    st = launch_status(launch_expert_weights(w, *dev, raw(stream)));
  }
  return st;
}

// Limits of a self-test of expired waits.
lt_status test_limits(int copied_tiles, unsigned int limit_us, RingLimits* ring) {
  if (copied_tiles < 0 || limit_us < 1 || limit_us > 1000000) return LT_ERR_INVALID_ARG;
  *ring = RingLimits{copied_tiles, static_cast<uint64_t>(limit_us) * 1000u};
  return LT_OK;
}

}  // namespace

extern "C" {

LT_API lt_status latent_tail_expert_gated(const uint16_t* x, const uint16_t* weights,
                                          const int32_t* offsets, uint16_t* hidden, void* saved,
                                          uint8_t* saved_exponents, int N, int E, int F, int C,
                                          lt_activation activation, lt_saved saved_kind,
                                          lt_stream stream) {
  return expert_gated(x, weights, offsets, hidden, saved, saved_exponents, N, E, F, C, activation,
                      saved_kind, RingLimits{}, stream);
}

LT_API lt_status latent_tail_selftest_expert_gated_timeout(
    const uint16_t* x, const uint16_t* weights, const int32_t* offsets, uint16_t* hidden,
    void* saved, uint8_t* saved_exponents, int N, int E, int F, int C, lt_activation activation,
    lt_saved saved_kind, int copied_tiles, unsigned int limit_us, lt_stream stream) {
  RingLimits ring;
  const lt_status st = test_limits(copied_tiles, limit_us, &ring);
  return st != LT_OK ? st
                     : expert_gated(x, weights, offsets, hidden, saved, saved_exponents, N, E, F, C,
                                    activation, saved_kind, ring, stream);
}

LT_API size_t latent_tail_expert_gated_backward_workspace_size(int N, int F) {
  if (N <= 0 || N > kMaxRows || F > kMaxWidth / 2 || check_width(F) != LT_OK) return 0;
  return bytes_of(N, 2 * static_cast<int64_t>(F), 2);
}

LT_API lt_status latent_tail_expert_gated_backward(
    const uint16_t* grad_hidden, const uint16_t* x, const uint16_t* weights, const void* saved,
    const uint8_t* saved_exponents, const int32_t* offsets, uint16_t* grad_x,
    uint16_t* grad_weights, uint16_t* hidden, int N, int E, int F, int C,
    lt_activation activation, lt_saved saved_kind, void* workspace, size_t workspace_bytes,
    lt_stream stream) {
  lt_status st = check_sizes(N, E, F, C, offsets);
  if (st != LT_OK) return st;
  if (F > kMaxWidth / 2 || !known(activation)) return LT_ERR_INVALID_ARG;
  if (saved_kind != LT_SAVED_BF16 && saved_kind != LT_SAVED_8BIT) return LT_ERR_INVALID_ARG;
  if (N == 0) return zero_weights(grad_weights, E, 2 * F, C, stream);
  if ((st = check_saved(saved_kind, saved, saved_exponents)) != LT_OK) return st;
  const bool products = grad_x != nullptr || grad_weights != nullptr;
  if (!products && hidden == nullptr) return LT_ERR_INVALID_ARG;
  if ((products && grad_hidden == nullptr) || (grad_x != nullptr && weights == nullptr) ||
      (grad_weights != nullptr && x == nullptr))
    return LT_ERR_INVALID_ARG;
  if ((st = check_optional({grad_hidden, x, weights, offsets, grad_x, grad_weights, hidden})) !=
      LT_OK)
    return st;
  const size_t need = products ? latent_tail_expert_gated_backward_workspace_size(N, F) : 0;
  if (need != 0) {
    if (workspace == nullptr || workspace_bytes < need) return LT_ERR_WORKSPACE;
    if (!aligned16(workspace)) return LT_ERR_ALIGNMENT;
  }
  const size_t w_bytes = E * bytes_of(2 * F, C, 2);
  if (!disjoint({span(grad_x, bytes_of(N, C, 2)), span(grad_weights, w_bytes),
                 span(hidden, bytes_of(N, F, 2)), span(need ? workspace : nullptr, need)},
                {span(grad_hidden, bytes_of(N, F, 2)), span(x, bytes_of(N, C, 2)),
                 span(weights, w_bytes), span(saved, saved_bytes(saved_kind, N, F)),
                 span(saved_exponents, bytes_of(N, 2, groups8(F))),
                 span(offsets, bytes_of(E + 1, 4, 1))}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev, Operator::kExperts)) != LT_OK) return st;
  uint16_t* pre = products ? static_cast<uint16_t*>(workspace) : nullptr;
  const GatedGradArgs g{grad_hidden, saved, saved_exponents, offsets, pre, hidden, N, E, F,
                        activation, saved_kind};
  if ((st = launch_status(launch_gated_grad(g, *dev, raw(stream)))) != LT_OK) return st;
  if (grad_x != nullptr) {
    const ExpertRowsArgs r{pre, weights, offsets, grad_x, N, E, C, 2 * F, true, RingLimits{}};
    if ((st = launch_status(launch_expert_rows(r, *dev, raw(stream)))) != LT_OK) return st;
  }
  if (grad_weights != nullptr) {
    const ExpertWeightsArgs w{pre, x, offsets, grad_weights, N, E, 2 * F, C, RingLimits{}};
    st = launch_status(launch_expert_weights(w, *dev, raw(stream)));
  }
  return st;
}

LT_API lt_status latent_tail_expert_matmul(const uint16_t* x, const uint16_t* weights,
                                           const int32_t* offsets, uint16_t* out, int N, int E,
                                           int M, int C, lt_stream stream) {
  return expert_matmul(x, weights, offsets, out, N, E, M, C, RingLimits{}, stream);
}

LT_API lt_status latent_tail_selftest_expert_matmul_timeout(
    const uint16_t* x, const uint16_t* weights, const int32_t* offsets, uint16_t* out, int N,
    int E, int M, int C, int copied_tiles, unsigned int limit_us, lt_stream stream) {
  RingLimits ring;
  const lt_status st = test_limits(copied_tiles, limit_us, &ring);
  return st != LT_OK ? st : expert_matmul(x, weights, offsets, out, N, E, M, C, ring, stream);
}

LT_API lt_status latent_tail_expert_matmul_backward(const uint16_t* grad_out, const uint16_t* x,
                                                    const uint16_t* weights,
                                                    const int32_t* offsets, uint16_t* grad_x,
                                                    uint16_t* grad_weights, int N, int E, int M,
                                                    int C, lt_stream stream) {
  return expert_matmul_backward(grad_out, x, weights, offsets, grad_x, grad_weights, N, E, M, C,
                                RingLimits{}, stream);
}

LT_API lt_status latent_tail_selftest_expert_matmul_backward_timeout(
    const uint16_t* grad_out, const uint16_t* x, const uint16_t* weights, const int32_t* offsets,
    uint16_t* grad_x, uint16_t* grad_weights, int N, int E, int M, int C, int copied_tiles,
    unsigned int limit_us, lt_stream stream) {
  RingLimits ring;
  const lt_status st = test_limits(copied_tiles, limit_us, &ring);
  return st != LT_OK ? st
                     : expert_matmul_backward(grad_out, x, weights, offsets, grad_x, grad_weights,
                                              N, E, M, C, ring, stream);
}

LT_API lt_status latent_tail_quantize8(const uint16_t* x, int8_t* values, uint8_t* exponents,
                                       int T, int C, lt_stream stream) {
  if (T < 0 || T > kMaxRows) return LT_ERR_INVALID_ARG;
  lt_status st = check_width(C);
  if (st != LT_OK || T == 0) return st;
  if ((st = check_ptrs({x, values, exponents})) != LT_OK) return st;
  if (!disjoint({span(values, bytes_of(T, C, 1)), span(exponents, bytes_of(T, groups8(C), 1))},
                {span(x, bytes_of(T, C, 2))}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != LT_OK) return st;
  const Quantize8Args a{x, values, exponents, nullptr, T, C};
  return launch_status(launch_quantize8(a, *dev, raw(stream)));
}

LT_API lt_status latent_tail_dequantize8(const int8_t* values, const uint8_t* exponents,
                                         uint16_t* out, int T, int C, lt_stream stream) {
  if (T < 0 || T > kMaxRows) return LT_ERR_INVALID_ARG;
  lt_status st = check_width(C);
  if (st != LT_OK || T == 0) return st;
  if ((st = check_ptrs({values, exponents, out})) != LT_OK) return st;
  if (!disjoint({span(out, bytes_of(T, C, 2))},
                {span(values, bytes_of(T, C, 1)), span(exponents, bytes_of(T, groups8(C), 1))}))
    return LT_ERR_INVALID_ARG;
  const lt::DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != LT_OK) return st;
  const Quantize8Args a{nullptr, const_cast<int8_t*>(values), const_cast<uint8_t*>(exponents), out,
                        T, C};
  return launch_status(launch_dequantize8(a, *dev, raw(stream)));
}

}  // extern "C"
