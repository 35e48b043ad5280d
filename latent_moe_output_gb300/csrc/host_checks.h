// Host-side argument checks and per-device state shared by the C-ABI layers
// (api.cu, block_api.cu). Not installed, not part of the ABI.
#pragma once

#include "latent_tail.h"
#include "launch.h"

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace lt {

// Operators whose kernels have attributes to set on a device before their first launch.
enum class Operator { kNone, kTail, kDispatch, kMatvec4, kResidualNorm, kExperts };

// Per-device state of the current device, set up on first use, with the kernels of `op`
// (those of an operator alone, so that no other pays for them or fails with them).
lt_status current_device(const DeviceInfo** out, Operator op = Operator::kNone);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  uintptr_t lo, hi;
};
inline Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes};
}
inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

inline lt_status check_ptrs(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p == nullptr) return LT_ERR_INVALID_ARG;
  for (const void* p : ptrs)
    if (!aligned16(p)) return LT_ERR_ALIGNMENT;
  return LT_OK;
}

inline size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

inline lt_status launch_status(cudaError_t e) { return e == cudaSuccess ? LT_OK : LT_ERR_CUDA; }

}  // namespace lt
