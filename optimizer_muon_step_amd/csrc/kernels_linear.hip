// Products of a layer's forward and input-gradient pass (see linear_gemm.h).
#include <hip/hip_runtime.h>

#include "linear_gemm.h"
#include "muon_internal.h"

namespace muon {

using namespace lin;

template <int TYPE, bool BKM>
static hipError_t launch_tile(const LinGemmArgs& a, int tile, hipStream_t s) {
  const int grid = a.tiles_m * a.tiles_n, threads = kLinTile[tile].threads;
  switch (tile) {  // tile, K slice, waves along m, n and k, stages, blocks to a compute unit
    case LIN_TILE_256: linear_gemm_kernel<TYPE, false, BKM, false, 256, 256, 64, 2, 4, 1, 2, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_128: linear_gemm_kernel<TYPE, false, BKM, false, 128, 128, 64, 2, 2, 1, 2, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64: linear_gemm_kernel<TYPE, false, BKM, false, 64, 64, 128, 2, 2, 2, 2, 2><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_64_DEEP: linear_gemm_kernel<TYPE, false, BKM, false, 64, 64, 128, 2, 1, 4, 4, 1><<<grid, threads, 0, s>>>(a); break;
    case LIN_TILE_32: linear_gemm_kernel<TYPE, false, BKM, false, 32, 64, 128, 1, 1, 4, 3, 2><<<grid, threads, 0, s>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_linear(const LinGemmArgs& a, int type, bool b_kmajor, int tile, hipStream_t s) {
  if (type == GRAD_BF16) return b_kmajor ? launch_tile<GRAD_BF16, true>(a, tile, s) : launch_tile<GRAD_BF16, false>(a, tile, s);
  return b_kmajor ? launch_tile<GRAD_FP16, true>(a, tile, s) : launch_tile<GRAD_FP16, false>(a, tile, s);
}

}  // namespace muon
