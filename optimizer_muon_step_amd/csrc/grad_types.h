// Kernel-argument tables of the gradient-norm, clipping and clipped-AdamW
// kernels, and their constants.  Plain C++ (no HIP headers): shared by the
// host code that fills the tables and the gfx950 kernels that read them.
//
// A call's pointers and sizes travel as kernel arguments, so it needs no
// table in device memory, no plan and no upload, and may be captured without
// an earlier call.  A launch takes as many tensors as fit KERNARG_BYTES;
// longer lists take several launches.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace muon {

constexpr int KERNARG_BYTES = 4096;
constexpr int GRAD_THREADS = 256;

enum GradType { GRAD_FP32 = 0, GRAD_BF16 = 1, GRAD_FP16 = 2 };
constexpr int grad_type_bytes(int t) { return t == GRAD_FP32 ? 4 : 2; }

// Work items of a launch are chunks of its tensors: tensor t owns items
// start[t] .. start[t + 1] - 1, all of the full chunk length except the last,
// whose elements are counted in tail[t] (shifted past the type bits).  A grid
// holds fewer than 2^32 threads, so a launch of one block per item takes
// fewer than 2^24 items.
constexpr int64_t MAX_LAUNCH_ITEMS = (1 << 24) - 1;
constexpr int64_t GRAD_MAX_NUMEL = (int64_t)1 << 35;

// ---- global norm ----
constexpr int NORM_CHUNK_BYTES = 16384;  // 4 x 16 bytes per thread
constexpr int NORM_MAX_BLOCKS = 1024;    // partial sums in the workspace
constexpr int NORM_GROUP = 32;           // blocks that count on one counter
constexpr int NORM_MAX_GROUPS = NORM_MAX_BLOCKS / NORM_GROUP;
constexpr int norm_chunk(int type) { return NORM_CHUNK_BYTES / grad_type_bytes(type); }

// The caller's workspace.  `arrived` counts the blocks of a group that have
// stored their partial sum, `groups` the groups that are complete; both are
// zero between calls.  Each counter has a 128-byte line of its own.
struct NormCounter {
  uint32_t arrived;
  uint32_t pad_[31];
};
struct NormWorkspace {
  NormCounter groups;
  NormCounter group[NORM_MAX_GROUPS];
  double part[NORM_MAX_BLOCKS];
};

constexpr int NORM_TENSORS = (KERNARG_BYTES - 64) / 16;
struct NormArgs {
  NormWorkspace* ws;
  float* record;        // {norm, factor}
  float max_norm, scale;
  int32_t n;            // tensors of this launch
  int32_t blocks;       // grid of every launch of the call
  int32_t first, last;  // first / last launch of the call
  int32_t start[NORM_TENSORS + 1];
  uint32_t tail[NORM_TENSORS];  // elements of the last chunk << 2 | type
  const void* p[NORM_TENSORS];
};
static_assert(sizeof(NormArgs) <= KERNARG_BYTES, "kernel arguments");

// ---- clipping ----
constexpr int CLIP_CHUNK = 8192;  // elements
constexpr int CLIP_TENSORS = (KERNARG_BYTES - 64) / 24;
struct ClipArgs {
  const float* record;
  int32_t n;
  int32_t items;
  int32_t start[CLIP_TENSORS + 1];
  uint32_t tail[CLIP_TENSORS];  // elements of the last chunk << 4 | output type << 2 | type
  const void* in[CLIP_TENSORS];
  void* out[CLIP_TENSORS];
};
static_assert(sizeof(ClipArgs) <= KERNARG_BYTES, "kernel arguments");

// ---- AdamW on clipped gradients ----
constexpr int ADAMC_CHUNK = 4096;  // elements
constexpr int ADAMC_DECAYS = 4;    // distinct weight decays of a launch
constexpr int ADAMC_TENSORS = (KERNARG_BYTES - 80) / 40;
struct AdamClipArgs {
  const float* record;  // {norm, factor}, or null: factor 1
  float lr, beta1, beta2, eps;
  float omb1, omb2;  // 1 - beta1, 1 - beta2
  float bc1, bc2;    // 1 - beta1^t, 1 - beta2^t
  float wd[ADAMC_DECAYS];
  int32_t n;
  int32_t items;
  int32_t start[ADAMC_TENSORS + 1];
  uint32_t tail[ADAMC_TENSORS];  // elements of the last chunk << 4 | decay index << 2 | gradient type
  float* p[ADAMC_TENSORS];
  const void* g[ADAMC_TENSORS];
  float* u[ADAMC_TENSORS];
  float* v[ADAMC_TENSORS];
};
static_assert(sizeof(AdamClipArgs) <= KERNARG_BYTES, "kernel arguments");

}  // namespace muon
