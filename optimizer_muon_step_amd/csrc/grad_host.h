// Host side of the gradient-norm, clipping and clipped-AdamW entry points
// that needs no GPU: argument validation and the split of a tensor list into
// launches.  Plain C++, built into libmuon.so and, with the host compiler
// alone, into a sanitizer build.
#pragma once

#include <stdint.h>

#include <vector>

#include "../../include/muon.h"
#include "grad_types.h"

namespace muon {

// ---- validation (every check runs before any device call) ----
int validate_grad_norm(const void* const* grads, const int64_t* numels, const int* types, int n, float max_norm,
                       float scale, const float* record, const void* workspace);
int validate_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* types,
                       const int* out_types, int n, float max_norm, float scale, const float* record,
                       const void* workspace);
int validate_adamw_clip(float* const* params, const void* const* grads, const int* types, float* const* u,
                        float* const* v, const int64_t* numels, const float* wd, int n, float lr, float beta1,
                        float beta2, float eps, int64_t step, const float* record);

// The record a Muon step reads against the arrays it writes.
int validate_step_record(float* const* params, float* const* moms, uint16_t* const* upd, const muon_shape_t* shapes,
                         int n, const float* record);

// ---- launch tables: pointers, items and flags; scalars are the caller's ----
// Tensors without elements take no part.  There is always at least one norm
// launch (it writes the record), all of one grid; the others may have none.
// Whether a norm or clip of these tensors is one small launch (outs and
// out_types null for a norm).
bool grad_small(const void* const* grads, void* const* outs, const int64_t* numels, const int* types,
                const int* out_types, int n, GradSmallArgs* out);
// keep_bytes: how much of the list's end the norm reads so as to stay cached.
std::vector<NormArgs> norm_launches(const void* const* grads, const int64_t* numels, const int* types, int n,
                                    int64_t keep_bytes);
std::vector<ClipArgs> clip_launches(const void* const* grads, void* const* outs, const int64_t* numels,
                                    const int* types, const int* out_types, int n);
std::vector<AdamClipArgs> adamw_clip_launches(float* const* params, const void* const* grads, const int* types,
                                              float* const* u, float* const* v, const int64_t* numels,
                                              const float* wd, int n);

}  // namespace muon
