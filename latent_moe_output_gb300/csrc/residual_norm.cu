// latent_tail_residual_norm and its gradient: the norm after a block, its gate,
// the scaled residual sum and the norm before the next block.
//
//   u = y * r1 * gp,  r1 = rsqrt(mean y^2 + eps)        (y itself without gp)
//   v = s * x + gate * u
//   z = v * r2 * gn,  r2 = rsqrt(mean v^2 + eps)
//
// Gradient, from dv (of v as an output) and dz:
//   a  = dz * gn,   d  = dv + r2 * (a - vh * mean(a * vh)),  vh = v * r2
//   dx = s * d,     dgate = d * u,   b = d * gate * gp
//   dy = r1 * (b - yh * mean(b * yh)),  yh = y * r1
//   dgp = sum_t d * gate * yh,  dgn = sum_t dz * vh
//
// Every element is read once and written once, so memory bounds both.
#include "block_launch.h"
#include "rows.cuh"

#include <algorithm>

namespace lt {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kReduceCols = 32;    // float4 columns per CTA of the column sum
constexpr int kReduceSlices = 16;  // parts of the partial rows per CTA

struct Shape {
  int threads;  // per CTA
  int tpr;      // threads per token row (whole warps)
  int per_cta;  // token rows a CTA works on at once
  int pieces;   // 8-element pieces per thread
};

Shape shape_of(int H) {
  const int nch = H / 8;
  Shape s;
  s.pieces = nch > kMaxThreads ? 2 : 1;
  if (nch <= 128) {
    s.tpr = nch <= 32 ? 32 : nch <= 64 ? 64 : 128;
    s.threads = 256;
  } else {
    s.tpr = std::min(kMaxThreads, (nch + 31) / 32 * 32);
    s.threads = s.tpr;
  }
  s.per_cta = s.threads / s.tpr;
  return s;
}

// Sum over the threads of a row. `red` holds one value per warp; consecutive
// calls alternate between two of them, so one barrier per call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int row_in_cta, int warps_per_row) {
  v = warp_sum_f(v);
  if (warps_per_row == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps_per_row; ++w) s += red[row_in_cta * warps_per_row + w];
  return s;
}

__device__ __forceinline__ void load8(const float* p, float (&a)[8]) {
  const float4 lo = __ldg(reinterpret_cast<const float4*>(p));
  const float4 hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
  a[0] = lo.x; a[1] = lo.y; a[2] = lo.z; a[3] = lo.w;
  a[4] = hi.x; a[5] = hi.y; a[6] = hi.z; a[7] = hi.w;
}

// Eight elements of the residual stream, bf16 or FP32.
template <bool kF32>
__device__ __forceinline__ void load_res8(const void* base, size_t at, float (&a)[8]) {
  if constexpr (kF32) {
    const float* p = static_cast<const float*>(base) + at;
    const uint4 lo = ld_once_v4(p), hi = ld_once_v4(p + 4);
    a[0] = __uint_as_float(lo.x); a[1] = __uint_as_float(lo.y);
    a[2] = __uint_as_float(lo.z); a[3] = __uint_as_float(lo.w);
    a[4] = __uint_as_float(hi.x); a[5] = __uint_as_float(hi.y);
    a[6] = __uint_as_float(hi.z); a[7] = __uint_as_float(hi.w);
  } else {
    unpack8(ld_once_v4(static_cast<const uint16_t*>(base) + at), a);
  }
}

template <bool kF32>
__device__ __forceinline__ void store_res8(void* base, size_t at, const float (&a)[8]) {
  if constexpr (kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(a[0], a[1], a[2], a[3]);
    p[1] = make_float4(a[4], a[5], a[6], a[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(a);
  }
}

__device__ __forceinline__ void gate8(const void* gate, int kind, int t, int col, size_t at,
                                      float (&a)[8]) {
  if (kind == kGateFull) {
    unpack8(ld_stream_v4(static_cast<const uint16_t*>(gate) + at), a);
  } else if (kind == kGateChannel) {
    load8(static_cast<const float*>(gate) + col, a);
  } else {
    const float g = kind == kGateToken ? __ldg(static_cast<const float*>(gate) + t) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = g;
  }
}

template <int kPieces, bool kF32>
__global__ void __launch_bounds__(kMaxThreads)
    residual_norm_kernel(const ResidualNormArgs a, int tpr) {
  __shared__ float red[2][kMaxThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int row = threadIdx.x / tpr, lane = threadIdx.x - row * tpr, wpr = tpr >> 5;
  const int t = blockIdx.x * (blockDim.x / tpr) + row;
  const bool live = t < a.T;
  const size_t base = static_cast<size_t>(t) * a.H;
  const float inv_h = 1.0f / static_cast<float>(a.H);

  float y[kPieces][8], x[kPieces][8], ss = 0.f;
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
    if (live && col < a.H) {
      const uint4 raw = ld_stream_v4(a.block + base + col);
      load_res8<kF32>(a.residual, base + col, x[q]);
      unpack8(raw, y[q]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[q][i] = y[q][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(y[q][i], y[q][i], ss);
  }
  float r1 = 1.f;
  if (a.post != nullptr) r1 = 1.0f / sqrtf(row_sum(ss, red[0], row, wpr) * inv_h + a.eps);
  ss = 0.f;
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
    if (live && col < a.H) {
      float w[8];
      if (a.post != nullptr) {
        load8(a.post + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[q][i] = y[q][i] * r1 * w[i];
      }
      gate8(a.gate, a.gate_kind, t, col, base + col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[q][i] = fmaf(w[i], y[q][i], a.scale * x[q][i]);
      store_res8<kF32>(a.residual_out, base + col, x[q]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[q][i], x[q][i], ss);
  }
  if (a.next == nullptr) return;
  const float r2 = 1.0f / sqrtf(row_sum(ss, red[1], row, wpr) * inv_h + a.eps);
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
    if (live && col < a.H) {
      float w[8];
      load8(a.next + col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = x[q][i] * r2 * w[i];
      *reinterpret_cast<uint4*>(a.next_out + base + col) = pack8(w);
    }
  }
}

// Each CTA walks over token rows and keeps the column sums of its threads'
// columns: in registers for one piece per thread, else in shared memory.
template <int kPieces, bool kF32>
__global__ void __launch_bounds__(kMaxThreads)
    residual_norm_backward_kernel(const ResidualNormBackwardArgs a, int tpr, int partial_rows) {
  extern __shared__ float s_acc[];  // kPieces > 1: [3][H]
  __shared__ float red[4][kMaxThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int row = threadIdx.x / tpr, lane = threadIdx.x - row * tpr, wpr = tpr >> 5;
  const int per_cta = blockDim.x / tpr;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  float acc[3][8] = {};
  if constexpr (kPieces > 1)
    for (int i = threadIdx.x; i < 3 * a.H; i += blockDim.x) s_acc[i] = 0.f;
  if constexpr (kPieces > 1) __syncthreads();
  auto add = [&](int which, int q, const float (&v)[8]) {
    if constexpr (kPieces == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[which][i] += v[i];
    } else {
      float* p = s_acc + static_cast<size_t>(which) * a.H + (lane + q * tpr) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] += v[i];
    }
  };

  for (int t0 = blockIdx.x * per_cta; t0 < a.T; t0 += gridDim.x * per_cta) {
    const int t = t0 + row;
    const bool live = t < a.T;
    const size_t base = static_cast<size_t>(t) * a.H;
    float y[kPieces][8], v[kPieces][8], d[kPieces][8], z[kPieces][8];
    float syy = 0.f, svv = 0.f, sav = 0.f;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int col = (lane + q * tpr) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[q][i] = v[q][i] = d[q][i] = z[q][i] = 0.f;
      if (live && col < a.H) {
        unpack8(ld_stream_v4(a.block + base + col), y[q]);
        load_res8<kF32>(a.residual_out, base + col, v[q]);
        if (a.grad_residual_out != nullptr) load_res8<kF32>(a.grad_residual_out, base + col, d[q]);
        if (a.next != nullptr) {
          float w[8];
          unpack8(ld_stream_v4(a.grad_next + base + col), z[q]);
          load8(a.next + col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            svv = fmaf(v[q][i], v[q][i], svv);
            sav = fmaf(z[q][i] * w[i], v[q][i], sav);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) syy = fmaf(y[q][i], y[q][i], syy);
    }
    float r1 = 1.f;
    if (a.post != nullptr) r1 = 1.0f / sqrtf(row_sum(syy, red[0], row, wpr) * inv_h + a.eps);
    if (a.next != nullptr) {
      const float r2 = 1.0f / sqrtf(row_sum(svv, red[1], row, wpr) * inv_h + a.eps);
      const float m = row_sum(sav, red[2], row, wpr) * inv_h * r2;  // mean(a * vh)
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int col = (lane + q * tpr) * 8;
        if (live && col < a.H) {
          float w[8];
          load8(a.next + col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float vh = v[q][i] * r2;
            d[q][i] = fmaf(r2, z[q][i] * w[i] - vh * m, d[q][i]);
            w[i] = z[q][i] * vh;
          }
          add(1, q, w);
        }
      }
    }
    float sgate = 0.f, sby = 0.f;
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int col = (lane + q * tpr) * 8;
      if (live && col < a.H) {
        float w[8], g[8], o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = a.scale * d[q][i];
        store_res8<kF32>(a.grad_residual, base + col, o);
        gate8(a.gate, a.gate_kind, t, col, base + col, g);
        if (a.post != nullptr) load8(a.post + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yh = y[q][i] * r1;
          const float u = a.post != nullptr ? yh * w[i] : y[q][i];
          o[i] = d[q][i] * u;
          sgate += o[i];
        }
        if (a.gate_kind == kGateChannel) add(2, q, o);
        if (a.gate_kind == kGateFull)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.grad_gate) + base + col) = pack8(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[q][i] *= g[i];
        if (a.post != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i] = d[q][i] * (y[q][i] * r1);
            d[q][i] *= w[i];
            sby = fmaf(d[q][i], y[q][i], sby);
          }
          add(0, q, o);
        }
      }
    }
    if (a.gate_kind == kGateToken) {
      sgate = row_sum(sgate, red[3], row, wpr);
      if (live && lane == 0) static_cast<float*>(a.grad_gate)[t] = sgate;
    }
    if (a.post != nullptr) {
      __syncthreads();
      const float m = row_sum(sby, red[0], row, wpr) * inv_h * r1;  // mean(b * yh)
#pragma unroll
      for (int q = 0; q < kPieces; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[q][i] = r1 * (d[q][i] - y[q][i] * r1 * m);
    }
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int col = (lane + q * tpr) * 8;
      if (live && col < a.H)
        *reinterpret_cast<uint4*>(a.grad_block + base + col) = pack8(d[q]);
    }
    __syncthreads();  // red is free for the next row
  }

  const size_t plane = static_cast<size_t>(partial_rows) * a.H;
  const size_t at = static_cast<size_t>(blockIdx.x * per_cta + row) * a.H;
  const bool want[3] = {a.post != nullptr, a.next != nullptr, a.gate_kind == kGateChannel};
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int col = (lane + q * tpr) * 8;
    if (col >= a.H) continue;
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      if (!want[s]) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = kPieces == 1 ? acc[s][i] : s_acc[static_cast<size_t>(s) * a.H + col + i];
      store_res8<true>(a.partials + s * plane, at + col, o);
    }
  }
}

// Sums of the partial rows, in a fixed order: 16 slices of rows per CTA, then
// the slices in order.
__global__ void __launch_bounds__(kReduceCols* kReduceSlices)
    column_sum_kernel(const float* __restrict__ partials, float* __restrict__ o0,
                      float* __restrict__ o1, float* __restrict__ o2, int partial_rows, int H) {
  __shared__ float4 s_part[kReduceSlices][kReduceCols];
  pdl_launch_dependents();
  pdl_wait();
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (out == nullptr) return;
  const int cx = threadIdx.x % kReduceCols, slice = threadIdx.x / kReduceCols;
  const int col = (blockIdx.x * kReduceCols + cx) * 4;
  const float* src = partials + blockIdx.y * static_cast<size_t>(partial_rows) * H + col;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H) {
#pragma unroll 4
    for (int r = slice; r < partial_rows; r += kReduceSlices) {
      const float4 v = *reinterpret_cast<const float4*>(src + static_cast<size_t>(r) * H);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  s_part[slice][cx] = s;
  __syncthreads();
  if (slice == 0 && col < H) {
    for (int i = 1; i < kReduceSlices; ++i) {
      const float4 v = s_part[i][cx];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    *reinterpret_cast<float4*>(out + col) = s;
  }
}

int backward_grid(int T, int H, int num_sms) {
  const Shape s = shape_of(H);
  const int ctas = std::max(1, 2048 / s.threads);  // resident threads per SM
  return std::max(1, std::min((T + s.per_cta - 1) / s.per_cta,
                              std::min(num_sms * (ctas > 2 ? 2 : ctas), 304)));
}

}  // namespace

int residual_norm_partial_rows(int T, int H) {
  return backward_grid(T, H, 304) * shape_of(H).per_cta;
}

cudaError_t setup_residual_norm(const DeviceInfo&) {
  const int bytes = 3 * 16384 * static_cast<int>(sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(residual_norm_backward_kernel<2, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(residual_norm_backward_kernel<2, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t launch_residual_norm(const ResidualNormArgs& a, const DeviceInfo&,
                                 cudaStream_t stream) {
  const Shape s = shape_of(a.H);
  const dim3 grid((a.T + s.per_cta - 1) / s.per_cta);
  auto* k = s.pieces == 1 ? (a.residual_f32 ? residual_norm_kernel<1, true>
                                            : residual_norm_kernel<1, false>)
                          : (a.residual_f32 ? residual_norm_kernel<2, true>
                                            : residual_norm_kernel<2, false>);
  return launch_dependent(k, grid, dim3(s.threads), 0, stream, a, s.tpr);
}

cudaError_t launch_residual_norm_backward(const ResidualNormBackwardArgs& a,
                                          const DeviceInfo& dev, cudaStream_t stream) {
  const Shape s = shape_of(a.H);
  const int grid = backward_grid(a.T, a.H, dev.num_sms);
  const int partial_rows = grid * s.per_cta;
  auto* k = s.pieces == 1 ? (a.residual_f32 ? residual_norm_backward_kernel<1, true>
                                            : residual_norm_backward_kernel<1, false>)
                          : (a.residual_f32 ? residual_norm_backward_kernel<2, true>
                                            : residual_norm_backward_kernel<2, false>);
  const size_t smem = s.pieces == 1 ? 0 : 3 * static_cast<size_t>(a.H) * sizeof(float);
  const cudaError_t e =
      launch_dependent(k, dim3(grid), dim3(s.threads), smem, stream, a, s.tpr, partial_rows);
  float* channel = a.gate_kind == kGateChannel ? static_cast<float*>(a.grad_gate) : nullptr;
  if (e != cudaSuccess || (a.post == nullptr && a.next == nullptr && channel == nullptr)) return e;
  const int cols = kReduceCols * 4;
  return launch_dependent(column_sum_kernel, dim3((a.H + cols - 1) / cols, 3),
                          dim3(kReduceCols * kReduceSlices), 0, stream,
                          static_cast<const float*>(a.partials), a.grad_post, a.grad_next_weight,
                          channel, partial_rows, a.H);
}

}  // namespace lt
