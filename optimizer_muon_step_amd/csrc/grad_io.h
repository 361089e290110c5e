// Gradient elements of the three types on gfx950: typed loads and stores of
// four at a time, and the search for an item's tensor in a launch's table.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bf16_util.h"
#include "grad_types.h"

namespace muon {
namespace grad {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// vec: four elements; wide: sixteen bytes, for passes that only read.  Both
// promise only their element's alignment: tensors may start anywhere in a flat
// buffer, and gfx950 loads and stores such vectors whole.
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint16_t u16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

template <int TYPE>
struct Elem;

template <>
struct Elem<GRAD_FP32> {
  typedef float scalar;
  typedef f32x4_u vec;
  typedef f32x4_u wide;
  static __device__ __forceinline__ f32x4 widen(vec w) { return f32x4{w.x, w.y, w.z, w.w}; }
  static __device__ __forceinline__ float widen1(scalar w) { return w; }
  static __device__ __forceinline__ vec narrow(f32x4 v) { return vec{v.x, v.y, v.z, v.w}; }
  static __device__ __forceinline__ scalar narrow1(float v) { return v; }
};

// 16-bit types: widening is exact; narrowing rounds once, to nearest even.
template <>
struct Elem<GRAD_BF16> {
  typedef uint16_t scalar;
  typedef u16x4_u vec;
  typedef u16x8_u wide;
  static __device__ __forceinline__ f32x4 widen(vec w) {
    return f32x4{bf16_bits_to_f32(w.x), bf16_bits_to_f32(w.y), bf16_bits_to_f32(w.z), bf16_bits_to_f32(w.w)};
  }
  static __device__ __forceinline__ float widen1(scalar w) { return bf16_bits_to_f32(w); }
  static __device__ __forceinline__ vec narrow(f32x4 v) {
    const uint32_t lo = pack_bf16x2(v.x, v.y), hi = pack_bf16x2(v.z, v.w);
    return vec{(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
  }
  static __device__ __forceinline__ scalar narrow1(float v) { return (uint16_t)f32_to_bf16_bits(v); }
};

template <>
struct Elem<GRAD_FP16> {
  typedef uint16_t scalar;
  typedef u16x4_u vec;
  typedef u16x8_u wide;
  static __device__ __forceinline__ f32x4 widen(vec w) {
    return __builtin_convertvector(__builtin_bit_cast(f16x4, u16x4{w.x, w.y, w.z, w.w}), f32x4);
  }
  static __device__ __forceinline__ float widen1(scalar w) { return (float)__builtin_bit_cast(_Float16, w); }
  static __device__ __forceinline__ vec narrow(f32x4 v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fp32_result(v[k]);
    const u16x4 h = __builtin_bit_cast(u16x4, __builtin_convertvector(v, f16x4));
    return vec{h.x, h.y, h.z, h.w};
  }
  static __device__ __forceinline__ scalar narrow1(float v) { return __builtin_bit_cast(uint16_t, (_Float16)fp32_result(v)); }
  // Keeps a product apart from its conversion: the compiler would otherwise
  // take both in one v_fma_mixlo_f16, whose product is not rounded to fp32.
  static __device__ __forceinline__ float fp32_result(float v) {
    asm("" : "+v"(v));
    return v;
  }
};

// The tensor that owns a work item, from a launch's table of first items
// (ascending from 0; START_UNUSED behind the last entry).  A wave holds the
// table in registers, so a search costs one trip to the kernel arguments and
// not one for each step of a bisection (norm of 61 tensors, 833 items: 8.6 -> 7.7 us).
// Every lane of the wave takes part; item is uniform over it.
template <int ENTRIES>
struct TensorFinder {
  static constexpr int K = (ENTRIES + 63) / 64;
  int32_t s[K];
  __device__ __forceinline__ explicit TensorFinder(const int32_t* start) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = k * 64 + lane < ENTRIES ? start[k * 64 + lane] : START_UNUSED;
  }
  // t with start[t] <= item < start[t + 1].
  __device__ __forceinline__ int operator()(int item) const {
    int c = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) c += __popcll(__ballot(s[k] <= item));
    return c - 1;
  }
  __device__ __forceinline__ int start_of(int t) const {
    int r = __builtin_amdgcn_readlane(s[0], t & 63);
#pragma unroll
    for (int k = 1; k < K; ++k) r = t >> 6 == k ? __builtin_amdgcn_readlane(s[k], t & 63) : r;
    return r;
  }
};

// f(Tag<type>) for a run-time element type.
template <int T>
struct Tag {
  static constexpr int value = T;
};
template <typename F>
__device__ __forceinline__ void with_type(int type, F&& f) {
  if (type == GRAD_FP32) f(Tag<GRAD_FP32>{});
  else if (type == GRAD_BF16) f(Tag<GRAD_BF16>{});
  else f(Tag<GRAD_FP16>{});
}

}  // namespace grad
}  // namespace muon
