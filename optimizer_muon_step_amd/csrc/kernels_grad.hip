// Global gradient norm and clipping on gfx950 (HBM-bound).
//
//   norm   = scale * sqrt(sum of g^2 over every element of every tensor)
//   factor = scale * min(1, max_norm / (norm + 1e-6))
//   out    = g * factor
//
// The sum is held in fp64 from the first square on: squares of fp32 values
// neither overflow nor underflow there, and its order is fixed, so the result
// is the same on every run.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bf16_util.h"
#include "grad_io.h"
#include "muon_internal.h"

namespace muon {

using namespace grad;

namespace {

constexpr int kWavesG = GRAD_THREADS / 64;

// Fixed-order block sum of one double per thread, valid in thread 0.
__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kWavesG; ++w) s += red[w];
  }
  return s;
}

// Sum of squares of this thread's elements of one chunk of len elements.
template <int TYPE>
__device__ __forceinline__ double chunk_squares(const void* base, int64_t off, int len) {
  typedef Elem<TYPE> E;
  constexpr int CH = norm_chunk(TYPE);
  constexpr int V = CH / (4 * GRAD_THREADS);
  const MUON_GLOBAL typename E::scalar* g = gptr(static_cast<const typename E::scalar*>(base)) + off;
  double s = 0.0;
  if (len == CH) {
    typename E::vec w[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
      w[k] = *reinterpret_cast<const MUON_GLOBAL typename E::vec*>(g + 4 * (k * GRAD_THREADS + threadIdx.x));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const f32x4 v = E::widen(w[k]);
      s += (double)v.x * v.x;
      s += (double)v.y * v.y;
      s += (double)v.z * v.z;
      s += (double)v.w * v.w;
    }
  } else {
    for (int e = threadIdx.x; e < len; e += GRAD_THREADS) {
      const double v = E::widen1(g[e]);
      s += v * v;
    }
  }
  return s;
}

}  // namespace

// Block b sums the squares of items b, b + blocks, ... and adds them to its
// partial in the workspace (the first launch of a call sets it).  In the last
// launch the block that arrives last sums all partials and writes the record.
__global__ __launch_bounds__(GRAD_THREADS) void grad_norm_kernel(const NormArgs a) {
  __shared__ double red[kWavesG];
  __shared__ int is_last;
  const int items = a.start[a.n];
  double s = 0.0;
  int t = 0;
  for (int it = blockIdx.x; it < items; it += a.blocks) {
    t = find_tensor(a.start, t, a.n, it);
    const uint32_t tail = a.tail[t];
    const int64_t c = it - a.start[t];
    const bool ends = it + 1 == a.start[t + 1];
    with_type(tail & 3, [&](auto tag) {
      constexpr int TYPE = decltype(tag)::value;
      s += chunk_squares<TYPE>(a.p[t], c * norm_chunk(TYPE), ends ? (int)(tail >> 2) : norm_chunk(TYPE));
    });
  }
  s = block_sum_f64(s, red);
  NormWorkspace* ws = a.ws;
  if (threadIdx.x == 0) {
    if (!a.first) s += ws->part[blockIdx.x];
    __hip_atomic_store(&ws->part[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    is_last = 0;
    if (a.last)
      is_last = __hip_atomic_fetch_add(&ws->arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.blocks - 1;
  }
  __syncthreads();
  if (!is_last) return;
  s = 0.0;
  for (int k = threadIdx.x; k < a.blocks; k += GRAD_THREADS)
    s += __hip_atomic_load(&ws->part[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = block_sum_f64(s, red);
  if (threadIdx.x == 0) {
    const double norm = (double)a.scale * sqrt(s);
    double c = 1.0;
    if (isnan(norm)) c = norm;
    else if (!isinf(a.max_norm)) c = fmin(1.0, (double)a.max_norm / (norm + 1e-6));
    a.record[0] = (float)norm;
    a.record[1] = (float)(a.scale * c);
    ws->arrived = 0;  // as the next call expects it
  }
}

namespace {

template <int TI, int TO>
__device__ __forceinline__ void clip_chunk(const void* in, void* out, int64_t off, int len, float factor) {
  typedef Elem<TI> I;
  typedef Elem<TO> O;
  constexpr int V = CLIP_CHUNK / (4 * GRAD_THREADS);
  const MUON_GLOBAL typename I::scalar* g = gptr(static_cast<const typename I::scalar*>(in)) + off;
  MUON_GLOBAL typename O::scalar* o = gptr(static_cast<typename O::scalar*>(out)) + off;
  if (len == CLIP_CHUNK) {
    typename I::vec w[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
      w[k] = *reinterpret_cast<const MUON_GLOBAL typename I::vec*>(g + 4 * (k * GRAD_THREADS + threadIdx.x));
#pragma unroll
    for (int k = 0; k < V; ++k)
      *reinterpret_cast<MUON_GLOBAL typename O::vec*>(o + 4 * (k * GRAD_THREADS + threadIdx.x)) =
          O::narrow(I::widen(w[k]) * factor);
  } else {
    for (int e = threadIdx.x; e < len; e += GRAD_THREADS) o[e] = O::narrow1(I::widen1(g[e]) * factor);
  }
}

}  // namespace

// One block per CLIP_CHUNK elements.  In place, a factor of 1 changes
// nothing, so those blocks end at once.
__global__ __launch_bounds__(GRAD_THREADS) void grad_clip_kernel(const ClipArgs a) {
  const int it = blockIdx.x;
  const float factor = a.record[1];
  const int t = find_tensor(a.start, 0, a.n, it);
  if (factor == 1.0f && a.in[t] == a.out[t]) return;
  const uint32_t tail = a.tail[t];
  const int64_t off = (int64_t)(it - a.start[t]) * CLIP_CHUNK;
  const int len = it + 1 == a.start[t + 1] ? (int)(tail >> 4) : CLIP_CHUNK;
  with_type(tail & 3, [&](auto ti) {
    with_type((tail >> 2) & 3, [&](auto to) {
      clip_chunk<decltype(ti)::value, decltype(to)::value>(a.in[t], a.out[t], off, len, factor);
    });
  });
}

hipError_t launch_grad_norm(const NormArgs& a, hipStream_t s) {
  grad_norm_kernel<<<a.blocks, GRAD_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t s) {
  if (a.items == 0) return hipSuccess;
  grad_clip_kernel<<<a.items, GRAD_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace muon
