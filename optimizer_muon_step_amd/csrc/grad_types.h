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
// whose elements are counted in tail[t] (shifted past the type bits); start
// holds START_UNUSED behind start[n].  A grid holds fewer than 2^32 threads,
// so a launch of one block per item takes fewer than 2^24 items.
constexpr int32_t START_UNUSED = INT32_MAX;
constexpr int64_t MAX_LAUNCH_ITEMS = (1 << 24) - 1;
constexpr int64_t GRAD_MAX_NUMEL = (int64_t)1 << 35;

// ---- global norm ----
constexpr int NORM_CHUNK_BYTES = 16384;  // 4 x 16 bytes per thread
constexpr int NORM_MAX_BLOCKS = 1024;    // partial sums in the workspace
// Gradients are read again by the clip or step that follows a norm: the last
// NORM_KEEP_BYTES of a call (the memory-side cache's size) are read with plain
// loads, which leave them in that cache, and what is before them with
// non-temporal ones, which are faster.  Measured with 0 and with 256 MiB
// kept: norm of 498 MB 75 and 79 us; norm and AdamW of 39.5 M elements 212
// and 191 us, of 124 M 644 and 617 us; norm and clip of 124 M bf16 elements
// into fp32 164 and 148 us.
constexpr int64_t NORM_KEEP_BYTES = (int64_t)256 << 20;
// A norm or clip of at most NORM_SMALL_ITEMS items (256 KB) is one launch of
// one block, a wave to an item: a norm takes 6.6 us a call against 7.3 by the
// other kernels, a clip 6.6 against 11.8, of 2 items, and 6.3 and 7.4, 7.5
// and 11.7 of 16.
constexpr int NORM_SMALL_ITEMS = 16;
constexpr int NORM_SMALL_THREADS = 1024;
constexpr int NORM_GROUP = 32;  // blocks that count on one counter
constexpr int NORM_MAX_GROUPS = NORM_MAX_BLOCKS / NORM_GROUP;
constexpr int norm_chunk(int type) { return NORM_CHUNK_BYTES / grad_type_bytes(type); }

// The caller's workspace.  `arrived` counts the blocks of a group that have
// stored their partial sum, `groups` the groups that are complete; both are
// zero between calls.  Counters are 128 bytes, a cache line, apart, so that no
// two share a line, whatever the alignment of the workspace.  Of the
// MUON_GRAD_WORKSPACE_BYTES that a caller gives the last 4224 are not used.
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
  int32_t n, items;     // tensors and work items of this launch
  int32_t blocks;       // grid of every launch of the call
  int32_t first, last;  // first / last launch of the call
  int32_t keep_from;    // items from here on are read so as to stay in the memory-side cache
  int32_t start[NORM_TENSORS + 1];
  uint32_t tail[NORM_TENSORS];  // elements of the last chunk << 2 | type
  const void* p[NORM_TENSORS];
};
static_assert(sizeof(NormArgs) <= KERNARG_BYTES, "kernel arguments");

// ---- clipping ----
// Out of place one block per item, in per-XCD runs of CLIP_RUN items; without
// the runs and with them, norm included: 1.56 G bf16 elements 1488 and 1466
// us, 124 M bf16 into fp32 152 and 149, 124 M fp32 228 and 227, 39.5 M fp32
// 73 and 74.  In place a factor of 1, the usual one, ends every block at
// once, and dispatching them is then all the time there is (1.3 ns each): at
// most CLIP_IN_PLACE_BLOCKS take the items in turn, which costs a long call
// that does clip 7 %.  With a block per item and with that many: 1.56 G bf16
// elements below the limit 542 and 470 us, clipped 1496 and 1607; 124 M fp32
// elements 83 and 80, 238 and 238.
constexpr int CLIP_CHUNK = 4096;  // elements
constexpr int CLIP_RUN = 64;
constexpr int CLIP_IN_PLACE_BLOCKS = 16384;
constexpr int CLIP_TENSORS = (KERNARG_BYTES - 64) / 24;
struct ClipArgs {
  const float* record;
  int32_t n;
  int32_t items;
  int32_t in_place;  // every out is its gradient
  int32_t start[CLIP_TENSORS + 1];
  uint32_t tail[CLIP_TENSORS];  // elements of the last chunk << 4 | output type << 2 | type
  const void* in[CLIP_TENSORS];
  void* out[CLIP_TENSORS];
};
static_assert(sizeof(ClipArgs) <= KERNARG_BYTES, "kernel arguments");

// ---- norm, or norm and clip, of a small call ----
struct GradSmallArgs {
  float* record;
  float max_norm, scale;
  int32_t n, items;
  int32_t start[NORM_SMALL_ITEMS + 1];
  uint32_t tail[NORM_SMALL_ITEMS];  // elements of the last chunk << 4 | output type << 2 | type
  const void* in[NORM_SMALL_ITEMS];
  void* out[NORM_SMALL_ITEMS];  // of a clip
};

// ---- AdamW on clipped gradients ----
// Elements per work item: long chunks, in per-XCD runs of ADAMC_LONG_RUN, for
// calls of at least ADAMC_LONG_MIN elements.  Measured with short and with
// long chunks, norm included: 39.5 M fp32 elements 192 and 202 us (fewer,
// larger blocks end less evenly), 124 M fp32 652 and 625 us, 1.56 G with bf16
// gradients 7.5 and 7.2 ms (7.3 without the runs).
constexpr int ADAMC_CHUNK = 4096, ADAMC_LONG_CHUNK = 8192;
constexpr int ADAMC_LONG_RUN = 16;
constexpr int64_t ADAMC_LONG_MIN = (int64_t)1 << 26;
constexpr int ADAMC_DECAYS = 4;  // distinct weight decays of a launch
constexpr int ADAMC_TENSORS = (KERNARG_BYTES - 80) / 40;
struct AdamClipArgs {
  const float* record;  // {norm, factor}, or null: factor 1
  float lr, beta1, beta2, eps;
  float omb1, omb2;  // 1 - beta1, 1 - beta2
  float bc1, bc2;    // 1 - beta1^t, 1 - beta2^t
  float wd[ADAMC_DECAYS];
  int32_t n;
  int32_t items;
  int32_t chunk;  // ADAMC_CHUNK or ADAMC_LONG_CHUNK
  int32_t start[ADAMC_TENSORS + 1];
  uint32_t tail[ADAMC_TENSORS];  // elements of the last chunk << 4 | decay index << 2 | gradient type
  float* p[ADAMC_TENSORS];
  const void* g[ADAMC_TENSORS];
  float* u[ADAMC_TENSORS];
  float* v[ADAMC_TENSORS];
};
static_assert(sizeof(AdamClipArgs) <= KERNARG_BYTES, "kernel arguments");

}  // namespace muon
