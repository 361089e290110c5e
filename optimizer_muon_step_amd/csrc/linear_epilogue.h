// Elements in groups of eight, activations, and the mask of dropout on gfx950:
// what the product kernels do to their sums before they store them, and what
// dropout does by itself.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16_util.h"
#include "grad_io.h"
#include "linear_types.h"

namespace muon {
namespace lin {

using grad::f32x4;
using grad::f32x4_u;

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight elements of a type, widened; any element alignment.
template <int TYPE>
__device__ __forceinline__ f32x8 widen8(u32x4 w) {
  if constexpr (TYPE == GRAD_BF16)
    return f32x8{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
  else
    return __builtin_convertvector(__builtin_bit_cast(f16x8, w), f32x8);
}
// Rounded once, to nearest even.
template <int TYPE>
__device__ __forceinline__ u32x4 narrow8(f32x8 v) {
  if constexpr (TYPE == GRAD_BF16) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
    // apart from the product or sum before: one v_fma_mix would round once where two roundings are meant
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = grad::Elem<GRAD_FP16>::fp32_result(v[k]);
    return __builtin_bit_cast(u32x4, __builtin_convertvector(v, f16x8));
  }
}

// 16 bytes of p from element i on.
template <int TYPE>
__device__ __forceinline__ u32x4 load_raw(const void* p, int64_t i) {
  const u32x4_u w = *reinterpret_cast<const MUON_GLOBAL u32x4_u*>(gptr(static_cast<const typename grad::Elem<TYPE>::scalar*>(p)) + i);
  return u32x4{w.x, w.y, w.z, w.w};
}

// Elements i .. i + 7 of p, or element i.
template <int TYPE>
__device__ __forceinline__ f32x8 load8(const void* p, int64_t i) {
  const MUON_GLOBAL typename grad::Elem<TYPE>::scalar* s = gptr(static_cast<const typename grad::Elem<TYPE>::scalar*>(p)) + i;
  if constexpr (TYPE == GRAD_FP32) {
    const f32x4_u lo = *reinterpret_cast<const MUON_GLOBAL f32x4_u*>(s), hi = *reinterpret_cast<const MUON_GLOBAL f32x4_u*>(s + 4);
    return f32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  } else {
    const u32x4_u w = *reinterpret_cast<const MUON_GLOBAL u32x4_u*>(s);
    return widen8<TYPE>(u32x4{w.x, w.y, w.z, w.w});
  }
}
template <int TYPE>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return grad::Elem<TYPE>::widen1(gptr(static_cast<const typename grad::Elem<TYPE>::scalar*>(p))[i]);
}

// The sum of eights `stride` apart, in their order; eight loads at a time.
__device__ __forceinline__ f32x8 sum_of_parts(const float* at, int64_t stride, int parts) {
  f32x8 v = load8<GRAD_FP32>(at, 0);
  for (int s = 1; s < parts; s += 8) {
    f32x8 more[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s + k < parts) more[k] = load8<GRAD_FP32>(at, (s + k) * stride);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s + k < parts) v += more[k];
  }
  return v;
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t i, f32x8 v) {
  MUON_GLOBAL typename grad::Elem<TYPE>::scalar* s = gptr(static_cast<typename grad::Elem<TYPE>::scalar*>(p)) + i;
  if constexpr (TYPE == GRAD_FP32) {
    *reinterpret_cast<MUON_GLOBAL f32x4_u*>(s) = f32x4_u{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<MUON_GLOBAL f32x4_u*>(s + 4) = f32x4_u{v[4], v[5], v[6], v[7]};
  } else {
    const u32x4 w = narrow8<TYPE>(v);
    *reinterpret_cast<MUON_GLOBAL u32x4_u*>(s) = u32x4_u{w.x, w.y, w.z, w.w};
  }
}
template <int TYPE>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  gptr(static_cast<typename grad::Elem<TYPE>::scalar*>(p))[i] = grad::Elem<TYPE>::narrow1(v);
}

// ---- activations ----
// The logistic function of 2u, u = sqrt(2/pi) (z + 0.044715 z^3): the tanh form
// of GELU is z / (1 + exp(-2u)), which keeps its relative accuracy where
// 1 + tanh(u) would cancel.  exp overflows to infinity for z below about -10, and
// the quotient is then -0.
constexpr float GELU_C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float GELU_C3 = 0.044715f;
constexpr float LOG2_E = 1.4426950408889634f;
__device__ __forceinline__ float gelu_exp(float z) {
  // exp(-2u) = 2^(z (c + c' z^2))
  return __builtin_amdgcn_exp2f(z * __builtin_fmaf(z * z, -GELU_C * GELU_C3 * LOG2_E, -GELU_C * LOG2_E));
}
// A comparison that is false for a NaN keeps it.
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == LIN_ACT_GELU) return z * __builtin_amdgcn_rcpf(1.0f + gelu_exp(z));
  if constexpr (ACT == LIN_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == LIN_ACT_RELU2) return z < 0.0f ? 0.0f : z * z;
  return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == LIN_ACT_GELU) {
    // s + z s (1 - s) 2u' with 1 - s = exp(-2u) s, which does not cancel.  Beyond
    // 10 the slope is within 1e-34 of 0 or 1, and exp or z^3 may overflow.
    const float t = gelu_exp(z), s = __builtin_amdgcn_rcpf(1.0f + t);
    const float v = __builtin_fmaf(z * s * (t * s), __builtin_fmaf(z * z, 3.0f * GELU_C3 * GELU_C, GELU_C), s);
    return z > 10.0f ? 1.0f : z < -10.0f ? 0.0f : v;
  }
  if constexpr (ACT == LIN_ACT_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);
  if constexpr (ACT == LIN_ACT_RELU2) return z < 0.0f ? 0.0f : 2.0f * z;
  return 1.0f;
}
// By an activation known at run time (uniform over the launch).
__device__ __forceinline__ float act_of(float z, int act) {
  if (act == LIN_ACT_GELU) return act_of<LIN_ACT_GELU>(z);
  if (act == LIN_ACT_RELU) return act_of<LIN_ACT_RELU>(z);
  return act == LIN_ACT_RELU2 ? act_of<LIN_ACT_RELU2>(z) : z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == LIN_ACT_GELU) return act_slope<LIN_ACT_GELU>(z);
  if (act == LIN_ACT_RELU) return act_slope<LIN_ACT_RELU>(z);
  return act == LIN_ACT_RELU2 ? act_slope<LIN_ACT_RELU2>(z) : 1.0f;
}
template <int ACT>
__device__ __forceinline__ f32x8 act8(f32x8 v) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = act_of<ACT>(v[k]);
  return v;
}
template <int ACT>
__device__ __forceinline__ f32x8 slope8(f32x8 z) {
#pragma unroll
  for (int k = 0; k < 8; ++k) z[k] = act_slope<ACT>(z[k]);
  return z;
}

// By an activation known at run time.
__device__ __forceinline__ f32x8 act8(f32x8 v, int act) {
  if (act == LIN_ACT_GELU) return act8<LIN_ACT_GELU>(v);
  if (act == LIN_ACT_RELU) return act8<LIN_ACT_RELU>(v);
  return act == LIN_ACT_RELU2 ? act8<LIN_ACT_RELU2>(v) : v;
}
__device__ __forceinline__ f32x8 slope8(f32x8 z, int act) {
  if (act == LIN_ACT_GELU) return slope8<LIN_ACT_GELU>(z);
  if (act == LIN_ACT_RELU) return slope8<LIN_ACT_RELU>(z);
  return slope8<LIN_ACT_RELU2>(z);
}

// ---- the mask ----
// 128 bits of the counter (group, row, site, step) under the key.
__device__ __forceinline__ u32x4 philox(uint32_t group, uint32_t row, uint32_t site, uint32_t step, uint32_t k0, uint32_t k1) {
  u32x4 c = {group, row, site, step};
#pragma unroll
  for (int r = 0; r < DROP_ROUNDS; ++r) {
    const uint64_t p0 = (uint64_t)c.x * 0xD2511F53u, p1 = (uint64_t)c.z * 0xCD9E8D57u;
    c = u32x4{(uint32_t)(p1 >> 32) ^ c.y ^ k0, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k1, (uint32_t)p0};
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The generator's key and step, of the launch or read from the device.
struct DropKey {
  uint32_t k0, k1, step;
  __device__ __forceinline__ explicit DropKey(const LinEpilogue& e) {
    uint64_t seed = e.seed;
    step = e.step;
    if (e.border != 0 && e.rng) {
      seed = (uint64_t)gptr(e.rng)[0];
      step = (uint32_t)gptr(e.rng)[1];
    }
    k0 = (uint32_t)seed;
    k1 = (uint32_t)(seed >> 32);
  }
};

// Eight elements at (row, col .. col + 7), col a multiple of 8, or one.  A
// dropped element is left out by a choice, not by a factor of 0: an infinity or
// NaN there does not reach the output.
__device__ __forceinline__ f32x8 drop8(const LinEpilogue& e, const DropKey& key, int64_t row, int64_t col, f32x8 v) {
  const u32x4 w = philox((uint32_t)(col >> 3), (uint32_t)row, e.site, key.step, key.k0, key.k1);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t bits = (k & 1) ? w[k >> 1] >> 16 : w[k >> 1] & 0xffffu;
    v[k] = bits >= e.border ? v[k] * e.keep_scale : 0.0f;
  }
  return v;
}
__device__ __forceinline__ float drop1(const LinEpilogue& e, const DropKey& key, int64_t row, int64_t col, float v) {
  const u32x4 w = philox((uint32_t)(col >> 3), (uint32_t)row, e.site, key.step, key.k0, key.k1);
  const int k = (int)col & 7;
  const uint32_t word = k < 4 ? (k < 2 ? w.x : w.y) : (k < 6 ? w.z : w.w);
  return ((k & 1) ? word >> 16 : word & 0xffffu) >= e.border ? v * e.keep_scale : 0.0f;
}

}  // namespace lin
}  // namespace muon
