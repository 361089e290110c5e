// Kernel arguments and constants of the hidden layers' products and of
// dropout.  Plain C++ (no HIP headers): shared by the host code that fills
// them in and the gfx950 kernels that read them.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "grad_types.h"

namespace muon {

enum LinAct { LIN_ACT_NONE = 0, LIN_ACT_GELU = 1, LIN_ACT_RELU = 2, LIN_ACT_RELU2 = 3 };

// The generator: Philox 4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC'11) with 7 rounds, the fewest that pass
// their whole test battery.  One call makes the 16 random bits of 8 elements.
constexpr int DROP_ROUNDS = 7;

// What is done to a product (or to a tensor, by muon_dropout) before it is
// stored; v is fp32 throughout and rounded once.
//   forward   z = v + bias;  [preact = z];  y = residual + drop(act(z))
//   backward  y = residual + drop(v) act'(preact)
struct LinEpilogue {
  const void* bias;  // of n elements, or null
  const void* residual;  // of y's type, or null
  void* y;
  void* preact;  // of the product's type; written forward, read backward; or null
  const int64_t* rng;  // {seed, step} on the device, or null
  int64_t ldr, ldy, ldp;
  uint64_t seed;
  uint32_t step, site;
  uint32_t border;  // elements whose 16 bits are below it are dropped; 0: no dropout
  float keep_scale;
  int32_t bias_type, y_type;
  int32_t act;
  int32_t backward;
};

// An operand as the products read it: 16-bit elements, 16-byte aligned, rows of
// a multiple of 8 elements apart, rows of a multiple of 8 elements.  64_ANY tiles read
// any other too (rows of 8 elements at least, B also fp32), and not by `bytes`.
struct LinOperand {
  const void* p;
  int64_t ld;     // bytes from row to row
  int64_t bytes;  // from p to the end of the last row
};

// Rows copied into such an operand, or rounded to its type.
struct LinPack {
  const void* src;
  void* dst;
  int64_t src_ld, dst_ld;  // elements; dst_ld is cols rounded up to 8, filled with zeros
  int64_t rows, cols;
  int32_t src_type, dst_type;
};
struct LinPackArgs {
  LinPack job[2];
  int32_t n;
};
constexpr int PACK_THREADS = 256;  // 8 elements each
constexpr int64_t pack_blocks(const LinPack& p) {
  return (p.rows * ((p.cols + 7) / 8) + PACK_THREADS - 1) / PACK_THREADS;
}

// `blocks` in launches of at most MAX_LAUNCH_ITEMS: f(first block, blocks), which gives 0, or
// what ends the sequence and is given back.
template <typename F>
int for_launches(int64_t blocks, F&& f) {
  for (int64_t first = 0; first < blocks; first += MAX_LAUNCH_ITEMS) {
    const int64_t left = blocks - first;
    if (const int rc = f(first, (int)(left < MAX_LAUNCH_ITEMS ? left : MAX_LAUNCH_ITEMS))) return rc;
  }
  return 0;
}

// One product C = A B, m x n over k.  Output tiles are numbered in groups of
// LIN_GROUP tile rows, column by column within a group, and each XCD takes a run
// of them: the 32 tiles that its compute units hold at a time then share 8
// row panels and 4 column panels in its L2.
constexpr int LIN_GROUP = 8;
struct LinGemmArgs {
  LinOperand a, b;
  int32_t m, n, k;
  int32_t tiles_m, tiles_n;
  int32_t slices;     // of K, of the tile's bk
  int32_t splits;     // of the slices; above 1 every split leaves its sums in part, split by split of (tiles_m BM) x (tiles_n BN)
  int32_t per_split;  // slices of a split
  LinEpilogue e;      // of the products of a layer
  // Of a weight gradient: C to c, or added to it; sums of the rows of dz (the B
  // operand's columns where sum_side is 1, the A operand's where it is 2) to
  // sums; with splits, sum_part holds splits x (the other side's tiles) x (sum_side's tiles x edge).
  float* c;
  float* sums;
  float* part;
  float* sum_part;
  int64_t ldc;
  int32_t add;
  int32_t sum_side;
};
static_assert(sizeof(LinGemmArgs) <= KERNARG_BYTES, "kernel arguments");

// c = [c +] the sums of the splits; likewise sums.
struct LinFinishArgs {
  float* c;
  float* sums;
  const float* part;
  const float* sum_part;
  int64_t ldc;
  int64_t part_ld, part_stride;          // of part, in elements
  int64_t sum_stride;                    // of sum_part
  int32_t m, n, n_sums;
  int32_t splits, sum_rows;              // rows of sum_part to add
  int32_t add;
  int32_t sum_first_block;               // blocks from here on take the sums
};
constexpr int FINISH_THREADS = 256, FINISH_SUMS = 32;  // sums of a block

// A layer's output from the sums of its splits.
struct LinJoinArgs {
  LinEpilogue e;
  const float* part;
  int64_t part_ld, part_stride;
  int32_t m, n, splits;
};
static_assert(sizeof(LinJoinArgs) <= KERNARG_BYTES, "kernel arguments");

// Output tiles of the product kernels (see kernels_linear.hip and linear_host.cpp).
// 64_DEEP and 32_DEEP have the whole LDS of a compute unit for their ring; 64_ANY loads through registers.
enum LinTile { LIN_TILE_256 = 0, LIN_TILE_256x192, LIN_TILE_128, LIN_TILE_64, LIN_TILE_64_DEEP, LIN_TILE_32, LIN_TILE_32_DEEP, LIN_TILE_64_ANY, LIN_TILES };
struct LinTileSize {
  int bm, bn, bk, threads;
};
constexpr LinTileSize kLinTile[LIN_TILES] = {
    {256, 256, 64, 512}, {256, 192, 64, 768}, {128, 128, 64, 256}, {64, 64, 128, 512}, {64, 64, 128, 512}, {32, 64, 128, 256}, {32, 64, 128, 256}, {64, 64, 128, 512}};

// Dropout by itself.
struct DropArgs {
  const void* x;
  int64_t ldx;
  int64_t m, n;
  int32_t x_type;
  LinEpilogue e;  // backward form, preact of x's type
};
constexpr int DROP_THREADS = 256;  // 8 elements each

}  // namespace muon
