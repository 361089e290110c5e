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
template <int WAVES>
__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += red[w];
  }
  return s;
}

// Sum of squares of this thread's elements (thread tid of THREADS) of one
// chunk of len elements; all its loads go out before the first square.  A
// partial chunk's vectors that fit are loaded whole, the up to 7 elements
// behind them one per thread.
template <int TYPE, bool FULL, bool KEEP, int THREADS>
__device__ __forceinline__ double chunk_squares(const void* base, int64_t off, int len, int tid) {
  typedef Elem<TYPE> E;
  constexpr int E16 = 16 / grad_type_bytes(TYPE);  // elements of a 16-byte load
  constexpr int V = norm_chunk(TYPE) / (E16 * THREADS);
  const MUON_GLOBAL typename E::scalar* g = gptr(static_cast<const typename E::scalar*>(base)) + off;
  typename E::wide w[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int e = E16 * (k * THREADS + tid);
    if (FULL || e + E16 <= len)
      w[k] = KEEP ? *reinterpret_cast<const MUON_GLOBAL typename E::wide*>(g + e)
                  : __builtin_nontemporal_load(reinterpret_cast<const MUON_GLOBAL typename E::wide*>(g + e));
    else
      w[k] = typename E::wide(0);
  }
  double s = 0.0;
  if (!FULL && tid < len % E16) {
    const double v = E::widen1(g[len - len % E16 + tid]);
    s = v * v;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int e = 0; e < E16; ++e) {
      const double v = E::widen1(w[k][e]);
      s += v * v;
    }
  return s;
}

// Writes the record of a call's sum of squares; returns the factor.
__device__ __forceinline__ float write_record(float* record, float max_norm, float scale, double sum) {
  const double norm = (double)scale * sqrt(sum);
  double c = 1.0;
  if (isnan(norm)) c = norm;
  else if (!isinf(max_norm)) c = fmin(1.0, (double)max_norm / (norm + 1e-6));
  record[0] = (float)norm;
  record[1] = (float)(scale * c);
  return (float)(scale * c);
}

typedef TensorFinder<NORM_TENSORS + 1> NormFinder;

// The block's items from it up to end; it moves on.
template <bool KEEP>
__device__ __forceinline__ double sum_items(const NormArgs& a, const NormFinder& find, int end, int& it) {
  double s = 0.0;
  for (; it < end; it += a.blocks) {
    const int t = find(it);
    const uint32_t tail = a.tail[t];
    const int64_t c = it - find.start_of(t);
    const bool ends = find(it + 1) != t;
    with_type(tail & 3, [&](auto tag) {
      constexpr int TYPE = decltype(tag)::value, CH = norm_chunk(TYPE);
      const int len = ends ? (int)(tail >> 2) : CH;
      if (len == CH) s += chunk_squares<TYPE, true, KEEP, GRAD_THREADS>(a.p[t], c * CH, CH, threadIdx.x);
      else s += chunk_squares<TYPE, false, KEEP, GRAD_THREADS>(a.p[t], c * CH, len, threadIdx.x);
    });
  }
  return s;
}

// Every load and store of this wave is complete: nothing moves across.
__device__ __forceinline__ void wait_memory() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("" ::: "memory");
}

// Counts one more arrival at c; whether it was the last of n, which leaves
// the counter at zero for the next call.
__device__ __forceinline__ bool arrive(NormCounter* c, int n) {
  const bool last = __hip_atomic_fetch_add(&c->arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)n - 1;
  if (last) __hip_atomic_store(&c->arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return last;
}

// Called by one thread of each block after its agent-scope stores.
__device__ __forceinline__ bool last_arrival(NormWorkspace* ws, int blocks) {
  const int groups = (blocks + NORM_GROUP - 1) / NORM_GROUP, g = blockIdx.x / NORM_GROUP;
  wait_memory();
  if (!arrive(&ws->group[g], min(NORM_GROUP, blocks - g * NORM_GROUP))) return false;
  return groups == 1 || arrive(&ws->groups, groups);
}

}  // namespace

// Bound by HBM reads: 498 MB in 79 us (6.3 TB/s), 3.1 GB of bf16 in 460 us
// (6.8 TB/s).
//
// Block b sums the squares of items b, b + blocks, ... and adds them to its
// partial in the workspace (the first launch of a call sets it).  In the last
// launch the block that arrives last sums all partials, in their order, and
// writes the record.
//
// Arrivals are counted per group of NORM_GROUP blocks and then over the
// groups: atomics on one address take 15 ns each, one after another.
// A partial is an agent-scope atomic store, complete at the coherence point
// before the block counts itself (the wait below), and the last block reads
// all of them with agent-scope atomic loads: no other memory passes between
// the blocks, so no cache needs writing back or invalidating (with
// acquire-release counting 1024 blocks take 37 us longer).
__global__ __launch_bounds__(GRAD_THREADS) void grad_norm_kernel(const NormArgs a) {
  __shared__ double red[kWavesG];
  __shared__ int is_last;
  const int items = a.items;
  const NormFinder find(a.start);
  int it = blockIdx.x;
  double s = sum_items<false>(a, find, min(items, a.keep_from), it);
  s += sum_items<true>(a, find, items, it);
  s = block_sum_f64<kWavesG>(s, red);
  NormWorkspace* ws = a.ws;
  if (threadIdx.x == 0) {
    if (!a.first) s += __hip_atomic_load(&ws->part[blockIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&ws->part[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    is_last = a.last && last_arrival(ws, a.blocks);
  }
  __syncthreads();
  if (!is_last) return;
  s = 0.0;
  for (int k = threadIdx.x; k < a.blocks; k += GRAD_THREADS)
    s += __hip_atomic_load(&ws->part[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  s = block_sum_f64<kWavesG>(s, red);
  if (threadIdx.x == 0) write_record(a.record, a.max_norm, a.scale, s);
}

namespace {

// One chunk of at most NORM_CHUNK_BYTES, held by one wave: whole 16-byte
// vectors as they are in memory, and the up to 7 elements behind them one per
// lane.  `rest` holds such an element widened.
constexpr int kHeld = NORM_CHUNK_BYTES / (16 * 64);
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
struct HeldChunk {
  u32x4_u w[kHeld];
  float rest;
};

// The vectors of a chunk of len elements of a type, and of those behind them.
struct HeldSize {
  int vectors, rest;
};
__device__ __forceinline__ HeldSize held_size(int type, int len) {
  const int e16 = 16 / grad_type_bytes(type);
  return {len / e16, len % e16};
}

template <int TI, int TO>
__device__ __forceinline__ void store_held(const HeldChunk& c, HeldSize n, void* out, int64_t off, float factor) {
  typedef Elem<TI> I;
  typedef Elem<TO> O;
  constexpr int E16 = 16 / grad_type_bytes(TI);
  MUON_GLOBAL typename O::scalar* o = gptr(static_cast<typename O::scalar*>(out)) + off;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    if (k * 64 + lane >= n.vectors) continue;
    const typename I::wide w = __builtin_bit_cast(typename I::wide, c.w[k]);
#pragma unroll
    for (int e = 0; e < E16; e += 4) {
      const f32x4 v = f32x4{I::widen1(w[e]), I::widen1(w[e + 1]), I::widen1(w[e + 2]), I::widen1(w[e + 3])} * factor;
      *reinterpret_cast<MUON_GLOBAL typename O::vec*>(o + E16 * (k * 64 + lane) + e) = O::narrow(v);
    }
  }
  if (lane < n.rest) o[E16 * n.vectors + lane] = O::narrow1(c.rest * factor);
}

}  // namespace

// A call of at most NORM_SMALL_ITEMS items: one block, a wave to an item,
// which it keeps in registers, so that a clip reads each gradient once and
// needs one launch, and the sum needs no partials in memory and no arrivals,
// whose trips to memory are most of a small call's time (norm of 8 tensors,
// 9984 fp32 elements: 3.3 us in the kernel, 4.8 in grad_norm_kernel).
template <bool CLIP>
__global__ __launch_bounds__(NORM_SMALL_THREADS) void grad_small_kernel(const GradSmallArgs a) {
  constexpr int kWaves = NORM_SMALL_THREADS / 64;
  static_assert(kWaves == NORM_SMALL_ITEMS, "one wave an item");
  __shared__ double red[kWaves];
  __shared__ float s_factor;
  const int it = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const bool mine = it < a.items;
  HeldChunk c;
  HeldSize n{0, 0};
  int t = 0, type = 0;
  int64_t off = 0;
  double s = 0.0;
  if (mine) {
    const TensorFinder<NORM_SMALL_ITEMS + 1> find(a.start);
    t = find(it);
    type = a.tail[t] & 3;
    const int chunk = norm_chunk(type);
    off = (int64_t)(it - find.start_of(t)) * chunk;
    n = held_size(type, find(it + 1) != t ? (int)(a.tail[t] >> 4) : chunk);
    const MUON_GLOBAL char* g = gptr(static_cast<const char*>(a.in[t])) + off * grad_type_bytes(type);
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      c.w[k] = k * 64 + lane < n.vectors ? *reinterpret_cast<const MUON_GLOBAL u32x4_u*>(g + 16 * (k * 64 + lane)) : u32x4_u(0);
    with_type(type, [&](auto tag) {
      typedef Elem<decltype(tag)::value> E;
      constexpr int E16 = 16 / grad_type_bytes(decltype(tag)::value);
      c.rest = 0.0f;
      if (lane < n.rest)
        c.rest = E::widen1(reinterpret_cast<const MUON_GLOBAL typename E::scalar*>(g)[E16 * n.vectors + lane]);
      s = (double)c.rest * c.rest;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const typename E::wide w = __builtin_bit_cast(typename E::wide, c.w[k]);
#pragma unroll
        for (int e = 0; e < E16; ++e) {
          const double v = E::widen1(w[e]);
          s += v * v;
        }
      }
    });
  }
  s = block_sum_f64<kWaves>(s, red);
  if (threadIdx.x == 0) s_factor = write_record(a.record, a.max_norm, a.scale, s);
  if (!CLIP) return;
  __syncthreads();
  const float factor = s_factor;
  if (!mine || (a.in[t] == a.out[t] && factor == 1.0f)) return;
  with_type(type, [&](auto ti) {
    with_type((a.tail[t] >> 2) & 3, [&](auto to) {
      store_held<decltype(ti)::value, decltype(to)::value>(c, n, a.out[t], off, factor);
    });
  });
}

namespace {

// Blocks of a clip launch.
__host__ __device__ __forceinline__ int clip_blocks(const ClipArgs& a) {
  return a.in_place && a.items > CLIP_IN_PLACE_BLOCKS ? CLIP_IN_PLACE_BLOCKS : a.items;
}

template <int TI, int TO, bool FULL>
__device__ __forceinline__ void clip_chunk(const void* in, void* out, int64_t off, int len, float factor) {
  typedef Elem<TI> I;
  typedef Elem<TO> O;
  constexpr int V = CLIP_CHUNK / (4 * GRAD_THREADS);
  const MUON_GLOBAL typename I::scalar* g = gptr(static_cast<const typename I::scalar*>(in)) + off;
  MUON_GLOBAL typename O::scalar* o = gptr(static_cast<typename O::scalar*>(out)) + off;
  typename I::vec w[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int e = 4 * (k * GRAD_THREADS + threadIdx.x);
    if (FULL || e + 4 <= len)
      w[k] = __builtin_nontemporal_load(reinterpret_cast<const MUON_GLOBAL typename I::vec*>(g + e));
  }
  if (!FULL && (int)threadIdx.x < len % 4) {
    const int e = len - len % 4 + threadIdx.x;
    o[e] = O::narrow1(I::widen1(g[e]) * factor);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int e = 4 * (k * GRAD_THREADS + threadIdx.x);
    if (FULL || e + 4 <= len)
      __builtin_nontemporal_store(O::narrow(I::widen(w[k]) * factor),
                                  reinterpret_cast<MUON_GLOBAL typename O::vec*>(o + e));
  }
}

}  // namespace

// One item is CLIP_CHUNK elements; block b takes items b, b + blocks, ... (one
// item each out of place).  In place a factor of 1 changes nothing.
//
// Bound by HBM.  Loads and stores are non-temporal: the gradients are read for
// the last time; with plain ones and so, norm included: 124 M bf16 elements
// into fp32 189 and 148 us (the second pass then moves 747 MB at 7.2 TB/s),
// as many fp32 ones 262 and 226, 39.5 M fp32 90 and 74.
__global__ __launch_bounds__(GRAD_THREADS) void grad_clip_kernel(const ClipArgs a) {
  const float factor = a.record[1];
  if (a.in_place && factor == 1.0f) return;
  const TensorFinder<CLIP_TENSORS + 1> find(a.start);
  const int blocks = clip_blocks(a);
  for (int b = blockIdx.x; b < a.items; b += blocks) {
    const int it = a.in_place ? b : ew_item_of_block(b, a.items, CLIP_RUN);
    const int t = find(it);
    if (a.in[t] == a.out[t] && factor == 1.0f) continue;
    const uint32_t tail = a.tail[t];
    const int64_t off = (int64_t)(it - find.start_of(t)) * CLIP_CHUNK;
    const int len = find(it + 1) != t ? (int)(tail >> 4) : CLIP_CHUNK;
    with_type(tail & 3, [&](auto ti) {
      with_type((tail >> 2) & 3, [&](auto to) {
        constexpr int TI = decltype(ti)::value, TO = decltype(to)::value;
        if (len == CLIP_CHUNK) clip_chunk<TI, TO, true>(a.in[t], a.out[t], off, len, factor);
        else clip_chunk<TI, TO, false>(a.in[t], a.out[t], off, len, factor);
      });
    });
  }
}

hipError_t launch_grad_norm(const NormArgs& a, hipStream_t s) {
  grad_norm_kernel<<<a.blocks, GRAD_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_small(const GradSmallArgs& a, bool clip, hipStream_t s) {
  if (clip)
    grad_small_kernel<true><<<1, NORM_SMALL_THREADS, 0, s>>>(a);
  else
    grad_small_kernel<false><<<1, NORM_SMALL_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ClipArgs& a, hipStream_t s) {
  if (a.items == 0) return hipSuccess;
  grad_clip_kernel<<<clip_blocks(a), GRAD_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace muon
