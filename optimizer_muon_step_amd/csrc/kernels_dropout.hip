// Dropout by itself and the copies that lay operands out on gfx950: passes
// over rows in groups of eight elements, HBM-bound.
#include <hip/hip_runtime.h>

#include "linear_epilogue.h"
#include "muon_internal.h"

namespace muon {

using namespace lin;

namespace {

// Where the eights of a block lie: eight i of the block, i below THREADS x
// CHUNKS, is at (row, 8 group).  One 64-bit division for a block; a thread's own
// is exact in fp32, since it divides less than 2^12 and is put right by one step.
struct Eights {
  int64_t row0;
  int64_t group0;
  int64_t per_row;
  __device__ __forceinline__ Eights(int64_t first, int64_t cols) {
    per_row = (cols + 7) >> 3;
    row0 = first / per_row;
    group0 = first - row0 * per_row;
  }
  __device__ __forceinline__ void at(int i, int64_t* row, int64_t* group) const {
    const int64_t g = group0 + i;
    if (per_row > 1024) {  // at most one row further
      const bool next = g >= per_row;
      *row = row0 + next;
      *group = next ? g - per_row : g;
      return;
    }
    const int n = (int)per_row, x = (int)g;
    int q = (int)((float)x * __builtin_amdgcn_rcpf((float)n));
    int r = x - q * n;
    if (r < 0) {
      --q;
      r += n;
    } else if (r >= n) {
      ++q;
      r -= n;
    }
    *row = row0 + q;
    *group = r;
  }
};

}  // namespace

// y = residual + drop(x) act'(preact).  Each thread has all of its loads out
// before it makes a mask; the last columns of a row that is no multiple of 8
// long are done one by one.
template <int XT, int YT, int ACT>
__global__ __launch_bounds__(DROP_THREADS) void dropout_kernel(const DropArgs a) {
  static_assert(DROP_THREADS * DROP_CHUNKS <= 1024, "see Eights");
  const LinEpilogue& e = a.e;
  const Eights eights((int64_t)blockIdx.x * (DROP_THREADS * DROP_CHUNKS), a.n);
  const DropKey key(e);
  int64_t row[DROP_CHUNKS], col[DROP_CHUNKS];
  bool whole[DROP_CHUNKS];
  f32x8 x[DROP_CHUNKS], z[DROP_CHUNKS], r[DROP_CHUNKS];
#pragma unroll
  for (int t = 0; t < DROP_CHUNKS; ++t) {
    eights.at(t * DROP_THREADS + threadIdx.x, &row[t], &col[t]);
    col[t] *= 8;
    whole[t] = row[t] < a.m && col[t] + 8 <= a.n;
    if (!whole[t]) continue;
    x[t] = load8<XT>(a.x, row[t] * a.ldx + col[t]);
    if constexpr (ACT != LIN_ACT_NONE) z[t] = load8<XT>(e.preact, row[t] * e.ldp + col[t]);
    if (e.residual) r[t] = load8<YT>(e.residual, row[t] * e.ldr + col[t]);
  }
#pragma unroll
  for (int t = 0; t < DROP_CHUNKS; ++t) {
    if (whole[t]) {
      f32x8 v = x[t];
      if constexpr (ACT != LIN_ACT_NONE) v = slope8<ACT>(z[t]) * v;
      if (e.border != 0) v = drop8(e, key, row[t], col[t], v);
      if (e.residual) v = r[t] + v;
      store8<YT>(e.y, row[t] * e.ldy + col[t], v);
    } else if (row[t] < a.m) {
#pragma unroll 1
      for (int64_t c = col[t]; c < a.n; ++c) {
        float v = load1<XT>(a.x, row[t] * a.ldx + c);
        if constexpr (ACT != LIN_ACT_NONE) v *= act_slope<ACT>(load1<XT>(e.preact, row[t] * e.ldp + c));
        if (e.border != 0) v = drop1(e, key, row[t], c, v);
        if (e.residual) v = load1<YT>(e.residual, row[t] * e.ldr + c) + v;
        store1<YT>(e.y, row[t] * e.ldy + c, v);
      }
    }
  }
}

template <int XT, int YT>
static hipError_t launch_dropout_of(const DropArgs& a, int grid, hipStream_t s) {
  switch (a.e.act) {
    case LIN_ACT_NONE: dropout_kernel<XT, YT, LIN_ACT_NONE><<<grid, DROP_THREADS, 0, s>>>(a); break;
    case LIN_ACT_GELU: dropout_kernel<XT, YT, LIN_ACT_GELU><<<grid, DROP_THREADS, 0, s>>>(a); break;
    case LIN_ACT_RELU: dropout_kernel<XT, YT, LIN_ACT_RELU><<<grid, DROP_THREADS, 0, s>>>(a); break;
    default: dropout_kernel<XT, YT, LIN_ACT_RELU2><<<grid, DROP_THREADS, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <int XT>
static hipError_t launch_dropout_from(const DropArgs& a, int grid, hipStream_t s) {
  if (a.e.y_type == GRAD_FP32) return launch_dropout_of<XT, GRAD_FP32>(a, grid, s);
  return a.e.y_type == GRAD_BF16 ? launch_dropout_of<XT, GRAD_BF16>(a, grid, s) : launch_dropout_of<XT, GRAD_FP16>(a, grid, s);
}

hipError_t launch_dropout(const DropArgs& a, int64_t blocks, hipStream_t s) {
  if (a.x_type == GRAD_FP32) return launch_dropout_from<GRAD_FP32>(a, (int)blocks, s);
  return a.x_type == GRAD_BF16 ? launch_dropout_from<GRAD_BF16>(a, (int)blocks, s) : launch_dropout_from<GRAD_FP16>(a, (int)blocks, s);
}

// Operands copied to rows that are aligned and a multiple of 8 long, with
// zeros behind their ends.
template <int ST, int DT>
__device__ __forceinline__ void pack_eight(const LinPack& p, int64_t row, int64_t col) {
  f32x8 v = 0.0f;
  if (col + 8 <= p.cols) {
    v = load8<ST>(p.src, row * p.src_ld + col);
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (col + k < p.cols) v[k] = load1<ST>(p.src, row * p.src_ld + col + k);
  }
  store8<DT>(p.dst, row * p.dst_ld + col, v);
}

__global__ __launch_bounds__(PACK_THREADS) void linear_pack_kernel(const LinPackArgs a, int blocks0) {
  static_assert(PACK_THREADS * PACK_CHUNKS <= 1024, "see Eights");
  const bool second = (int)blockIdx.x >= blocks0;
  const LinPack& p = a.job[second];
  const Eights eights((int64_t)((int)blockIdx.x - (second ? blocks0 : 0)) * (PACK_THREADS * PACK_CHUNKS), p.cols);
#pragma unroll
  for (int t = 0; t < PACK_CHUNKS; ++t) {
    int64_t row, group;
    eights.at(t * PACK_THREADS + threadIdx.x, &row, &group);
    if (row >= p.rows) continue;
    if (p.src_type != GRAD_FP32)
      pack_eight<GRAD_BF16, GRAD_BF16>(p, row, group * 8);  // either 16-bit type: the widened bits go back as they were
    else if (p.dst_type == GRAD_BF16)
      pack_eight<GRAD_FP32, GRAD_BF16>(p, row, group * 8);
    else
      pack_eight<GRAD_FP32, GRAD_FP16>(p, row, group * 8);
  }
}

hipError_t launch_linear_pack(const LinPackArgs& a, hipStream_t s) {
  const int64_t b0 = pack_blocks(a.job[0]), b1 = a.n > 1 ? pack_blocks(a.job[1]) : 0;
  linear_pack_kernel<<<(int)(b0 + b1), PACK_THREADS, 0, s>>>(a, (int)b0);
  return hipGetLastError();
}

}  // namespace muon
