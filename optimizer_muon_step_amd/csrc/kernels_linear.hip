// Products of a layer's forward and input-gradient pass (see linear_gemm.h).
#include <hip/hip_runtime.h>

#include "linear_gemm.h"
#include "muon_internal.h"

namespace muon {

using namespace lin;

template <int TYPE, bool BKM>
static hipError_t launch_tile(const LinGemmArgs& a, int tile, bool b_wide, hipStream_t s) {
  const int grid = a.tiles_m * a.tiles_n * a.splits, threads = kLinTile[tile].threads;
  switch (tile) {  // tile, K slice, waves along m, n and k, stages, blocks to a compute unit
    case LIN_TILE_256: linear_gemm_kernel<TYPE, false, BKM, false, 256, 256, 64, 2, 4, 1, 2, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_256x192: linear_gemm_kernel<TYPE, false, BKM, false, 256, 192, 64, 4, 3, 1, 2, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_128: linear_gemm_kernel<TYPE, false, BKM, false, 128, 128, 64, 2, 2, 1, 2, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64: linear_gemm_kernel<TYPE, false, BKM, false, 64, 64, 128, 2, 2, 2, 2, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64_DEEP: linear_gemm_kernel<TYPE, false, BKM, false, 64, 64, 128, 2, 1, 4, 4, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_32: linear_gemm_kernel<TYPE, false, BKM, false, 32, 64, 128, 1, 1, 4, 3, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_32_DEEP: linear_gemm_kernel<TYPE, false, BKM, false, 32, 64, 128, 1, 1, 4, 6, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64_ANY:
      if (b_wide) linear_gemm_kernel<TYPE, false, BKM, false, 64, 64, 128, 2, 2, 2, 2, 2, READ_ANY_WIDE><<<grid, threads, 0, s>>>(a);
      else linear_gemm_kernel<TYPE, false, BKM, false, 64, 64, 128, 2, 2, 2, 2, 2, READ_ANY><<<grid, threads, 0, s>>>(a);
      break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// The output of a product whose K was split: a thread to eight elements.  The
// splits are added in their order, so equal calls give equal bits.  Latency: one load of
// all splits up to 8, then the epilogue; about 3 us with the launch.
template <int TYPE>
__global__ __launch_bounds__(FINISH_THREADS) void linear_join_kernel(const LinJoinArgs a) {
  const int eights = (a.n + 7) >> 3;
  const int64_t i = (int64_t)blockIdx.x * FINISH_THREADS + threadIdx.x;
  const int64_t row = i / eights;
  if (row >= a.m) return;
  const int col = (int)(i - row * eights) * 8, have = min(8, a.n - col);
  // the rows of part are padded to whole tiles
  const f32x8 v = sum_of_parts(a.part + row * a.part_ld + col, a.part_stride, a.splits);
  const DropKey key(a.e);
  const LayerEdge<TYPE> store = {a.e, key};
  if (have == 8) {
    store.eight(row, col, v);
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < have) store.one(row, col + k, v[k]);
  }
}

hipError_t launch_linear_join(const LinJoinArgs& a, int type, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.m * ((a.n + 7) / 8) + FINISH_THREADS - 1) / FINISH_THREADS;
  if (type == GRAD_BF16) linear_join_kernel<GRAD_BF16><<<(int)blocks, FINISH_THREADS, 0, s>>>(a);
  else linear_join_kernel<GRAD_FP16><<<(int)blocks, FINISH_THREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear(const LinGemmArgs& a, int type, bool b_kmajor, bool b_wide, int tile, hipStream_t s) {
  if (type == GRAD_BF16)
    return b_kmajor ? launch_tile<GRAD_BF16, true>(a, tile, b_wide, s) : launch_tile<GRAD_BF16, false>(a, tile, b_wide, s);
  return b_kmajor ? launch_tile<GRAD_FP16, true>(a, tile, b_wide, s) : launch_tile<GRAD_FP16, false>(a, tile, b_wide, s);
}

}  // namespace muon
