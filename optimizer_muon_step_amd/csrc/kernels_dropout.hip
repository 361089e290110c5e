// Dropout by itself and the copies that lay operands out on gfx950: passes
// over rows in groups of eight elements, HBM-bound.
#include <hip/hip_runtime.h>

#include "linear_epilogue.h"
#include "muon_internal.h"

namespace muon {

using namespace lin;

namespace {

// Where a thread's eight lies: at (row, col), `have` of its elements within the rows
// of `cols`.  One 64-bit division for a block; a thread's own is exact in fp32, since
// what it divides is below 2^11, and is put right by one step.
struct Eight {
  int64_t row, col;
  int have;
  __device__ __forceinline__ Eight(int64_t first, int i, int64_t rows, int64_t cols) {
    const int64_t per_row = (cols + 7) >> 3;
    row = first / per_row;
    int64_t group = first - row * per_row + i;
    if (per_row >= 1024) {  // at most one row further
      const bool next = group >= per_row;
      row += next;
      group -= next ? per_row : 0;
    } else {
      const int n = (int)per_row, x = (int)group;
      int q = (int)((float)x * __builtin_amdgcn_rcpf((float)n));
      int r = x - q * n;
      if (r < 0) {
        --q;
        r += n;
      } else if (r >= n) {
        ++q;
        r -= n;
      }
      row += q;
      group = r;
    }
    col = group * 8;
    have = row < rows ? (int)min((int64_t)8, cols - col) : 0;
  }
};

}  // namespace

// Elements i .. i + 7 of p, the first `have` of them (the others as zeros).
template <int TYPE>
__device__ __forceinline__ f32x8 load_some(const void* p, int64_t i, int have) {
  if (have >= 8) return load8<TYPE>(p, i);
  f32x8 v = 0.0f;
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < have) v[k] = load1<TYPE>(p, i + k);
  return v;
}

// y = residual + drop(x) act'(preact), an eight to a thread: 16384 x 768 bf16 with a
// residual 13.6 us where three sets of operands, 226 MB, change places in the 256 MiB memory-side
// cache (5.5 TB/s; the generator's 7 rounds hide behind the loads), with two 14.0 and with four 15.5;
// 17.4 us (4.3 TB/s) where 12 sets leave nothing in it.  Loads or stores past the caches gained nothing.
template <int XT, int YT, int ACT>
__global__ __launch_bounds__(DROP_THREADS) void dropout_kernel(const DropArgs a) {
  const LinEpilogue& e = a.e;
  const Eight at((int64_t)blockIdx.x * DROP_THREADS, threadIdx.x, a.m, a.n);
  if (at.have == 0) return;
  const DropKey key(e);
  f32x8 v = load_some<XT>(a.x, at.row * a.ldx + at.col, at.have), z, r;
  if constexpr (ACT != LIN_ACT_NONE) z = load_some<XT>(e.preact, at.row * e.ldp + at.col, at.have);
  if (e.residual) r = load_some<YT>(e.residual, at.row * e.ldr + at.col, at.have);
  if constexpr (ACT != LIN_ACT_NONE) v = slope8<ACT>(z) * v;
  if (e.border != 0) v = drop8(e, key, at.row, at.col, v);
  if (e.residual) v = r + v;
  const int64_t y = at.row * e.ldy + at.col;
  if (at.have >= 8) {
    store8<YT>(e.y, y, v);
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < at.have) store1<YT>(e.y, y + k, v[k]);
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
// zeros behind their ends; an eight to a thread, in several launches where a grid cannot hold
// the blocks.  1999 x 1001 fp16 and 1001 x 771 fp32, 12 MB in all, 6.4 us.
__global__ __launch_bounds__(PACK_THREADS) void linear_pack_kernel(const LinPackArgs a, int64_t blocks0, int64_t first) {
  const int64_t block = first + blockIdx.x;
  const bool second = block >= blocks0;
  const LinPack& p = a.job[second];
  const Eight at((block - (second ? blocks0 : 0)) * PACK_THREADS, threadIdx.x, p.rows, p.cols);
  if (at.have == 0) return;
  const int64_t src = at.row * p.src_ld + at.col, dst = at.row * p.dst_ld + at.col;
  if (p.src_type != GRAD_FP32)  // either 16-bit type: the widened bits go back as they were
    store8<GRAD_BF16>(p.dst, dst, load_some<GRAD_BF16>(p.src, src, at.have));
  else if (p.dst_type == GRAD_BF16)
    store8<GRAD_BF16>(p.dst, dst, load_some<GRAD_FP32>(p.src, src, at.have));
  else
    store8<GRAD_FP16>(p.dst, dst, load_some<GRAD_FP32>(p.src, src, at.have));
}

hipError_t launch_linear_pack(const LinPackArgs& a, hipStream_t s) {
  const int64_t b0 = pack_blocks(a.job[0]), b1 = a.n > 1 ? pack_blocks(a.job[1]) : 0;
  return (hipError_t)for_launches(b0 + b1, [&](int64_t first, int blocks) {
    linear_pack_kernel<<<blocks, PACK_THREADS, 0, s>>>(a, b0, first);
    return (int)hipGetLastError();
  });
}

}  // namespace muon
