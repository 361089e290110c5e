// Host side of the hidden layers' products and of dropout that needs no GPU:
// argument validation, the choice of kernel and the kernels' arguments.  Plain
// C++, built into libmuon.so and, with the host compiler alone, into a
// sanitizer build.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/muon.h"
#include "linear_types.h"

namespace muon {

// The launches of one product.  Operands that the kernels cannot read where
// they are go to the workspace first; with splits a last pass adds them up.
struct LinPlan {
  bool empty;      // nothing to compute
  bool b_kmajor;   // of a layer's product (a weight gradient's operands both are)
  bool b_wide;     // B is read as fp32
  int type;
  int tile;
  LinPackArgs pack;  // n of 0: nothing to copy
  LinGemmArgs gemm;
  bool finish;         // K was split: a last pass adds the sums up, by
  LinFinishArgs fin;   // of a weight gradient
  LinJoinArgs join;    // of a layer
  size_t workspace;  // bytes; with a null workspace the pointers into it are offsets
};

// A layer's product, forward or (backward) for the gradient of its input.
// Every check runs before any device call.
int plan_linear(const muon_linear_t* l, bool backward, void* workspace, size_t workspace_bytes, LinPlan* out);
int plan_linear_dw(const muon_linear_dw_t* l, void* workspace, size_t workspace_bytes, LinPlan* out);

// Blocks of the launch in *blocks, 0 where there is nothing to do.
int plan_dropout(const muon_dropout_t* d, DropArgs* out, int64_t* blocks);

// Bytes of workspace; checks sizes, types and the distances of what is read, not pointers.
int linear_workspace(const muon_linear_t* l, bool backward, size_t* bytes);
int linear_dw_workspace(const muon_linear_dw_t* l, size_t* bytes);

}  // namespace muon
