// Weight-gradient products of a layer (see linear_gemm.h) and the pass that
// adds the splits of a long reduction.
#include <hip/hip_runtime.h>

#include "linear_gemm.h"
#include "muon_internal.h"

namespace muon {

using namespace lin;

template <int TYPE>
static hipError_t launch_tile(const LinGemmArgs& a, int tile, hipStream_t s) {
  const int grid = a.tiles_m * a.tiles_n * a.splits, threads = kLinTile[tile].threads;
  switch (tile) {  // as in kernels_linear.hip
    case LIN_TILE_256: linear_gemm_kernel<TYPE, true, true, true, 256, 256, 64, 2, 4, 1, 2, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_256x192: linear_gemm_kernel<TYPE, true, true, true, 256, 192, 64, 4, 3, 1, 2, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_128: linear_gemm_kernel<TYPE, true, true, true, 128, 128, 64, 2, 2, 1, 2, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64: linear_gemm_kernel<TYPE, true, true, true, 64, 64, 128, 2, 2, 2, 2, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64_ANY: linear_gemm_kernel<TYPE, true, true, true, 64, 64, 128, 2, 2, 2, 2, 2, READ_ANY><<<grid, threads, 0, s>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_linear_dw(const LinGemmArgs& a, int type, int tile, hipStream_t s) {
  return type == GRAD_BF16 ? launch_tile<GRAD_BF16>(a, tile, s) : launch_tile<GRAD_FP16>(a, tile, s);
}

// A thread to eight elements of a row of c, and behind them a block to 32 of the
// sums, whose many rows its 8 groups of threads share.  Everything is added in an order
// that the sizes give, so equal calls give equal bits.  Memory-bound: 5 splits of 768 x 3072
// added to c, 66 MB, 11.8 us (5.6 TB/s, more than HBM's 5.1: the launch before has just written
// the 47 MB of parts, which the memory-side cache holds).
__global__ __launch_bounds__(FINISH_THREADS) void linear_finish_kernel(const LinFinishArgs a) {
  if ((int)blockIdx.x >= a.sum_first_block) {
    constexpr int GROUPS = FINISH_THREADS / FINISH_SUMS;
    __shared__ float of_group[GROUPS][FINISH_SUMS];
    const int lane = threadIdx.x % FINISH_SUMS, group = threadIdx.x / FINISH_SUMS;
    const int i = ((int)blockIdx.x - a.sum_first_block) * FINISH_SUMS + lane;
    const MUON_GLOBAL float* p = gptr(a.sum_part) + min(i, a.n_sums - 1);
    float v = 0.0f;
    for (int r = group; r < a.sum_rows; r += 4 * GROUPS) {
      float more[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) more[k] = r + k * GROUPS < a.sum_rows ? p[(r + k * GROUPS) * a.sum_stride] : 0.0f;
      v += (more[0] + more[1]) + (more[2] + more[3]);
    }
    of_group[group][lane] = v;
    __syncthreads();
    if (group != 0 || i >= a.n_sums) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) v += of_group[g][lane];
    gptr(a.sums)[i] = a.add ? gptr(a.sums)[i] + v : v;
    return;
  }
  const int eights = (a.n + 7) >> 3;
  const int64_t i = (int64_t)blockIdx.x * FINISH_THREADS + threadIdx.x;
  const int64_t row = i / eights;
  if (row >= a.m) return;
  const int col = (int)(i - row * eights) * 8, have = min(8, a.n - col);
  // the rows of part are padded to whole tiles
  const f32x8 v = sum_of_parts(a.part + row * a.part_ld + col, a.part_stride, a.splits);
  const GradEdge store = {a.c, a.ldc, a.add != 0};
  if (have == 8) {
    store.eight(row, col, v);
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < have) store.one(row, col + k, v[k]);
  }
}

hipError_t launch_linear_finish(const LinFinishArgs& a, hipStream_t s) {
  const int blocks = a.sum_first_block + (a.n_sums + FINISH_SUMS - 1) / FINISH_SUMS;
  linear_finish_kernel<<<blocks, FINISH_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace muon
