// C ABI of the gradient norm, clipping and AdamW on clipped gradients: each
// call validates on the host and enqueues its launches; pointers and sizes
// travel as kernel arguments, so nothing is cached or allocated on the device.
#include <hip/hip_runtime.h>

#include <cmath>
#include <mutex>
#include <vector>

#include "../../include/muon.h"
#include "api_internal.h"
#include "grad_host.h"
#include "muon_internal.h"

namespace muon {
namespace {

// The launches of a norm, enqueued without another call's in between (the
// caller holds api_mutex()).
int enqueue_norm(std::vector<NormArgs>& launches, float max_norm, float scale, float* record, void* workspace,
                 hipStream_t stream) {
  for (NormArgs& a : launches) {
    a.ws = static_cast<NormWorkspace*>(workspace);
    a.record = record;
    a.max_norm = max_norm;
    a.scale = scale;
    const int rc = timed(MUON_KERNEL_GRAD_NORM, stream, [&] { return launch_grad_norm(a, stream); },
                         "gradient norm kernel launch");
    if (rc) return rc;
  }
  return MUON_OK;
}

// The one launch of a small norm, or of a small clip with its norm (timed as
// the clip).
int enqueue_small(GradSmallArgs& a, bool clip, float max_norm, float scale, float* record, hipStream_t stream) {
  a.record = record;
  a.max_norm = max_norm;
  a.scale = scale;
  std::lock_guard<std::mutex> lock(api_mutex());
  return timed(clip ? MUON_KERNEL_GRAD_CLIP : MUON_KERNEL_GRAD_NORM, stream,
               [&] { return launch_grad_small(a, clip, stream); }, "gradient norm kernel launch");
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_grad_norm(const void* const* grads, const int64_t* numels, const int* dtypes, int n, float max_norm,
                   float scale, float* record, void* workspace, hipStream_t stream) {
  return c_entry([&] {
    clear_error();
    const int rc = validate_grad_norm(grads, numels, dtypes, n, max_norm, scale, record, workspace);
    if (rc) return rc;
    GradSmallArgs small;
    if (grad_small(grads, nullptr, numels, dtypes, nullptr, n, &small))
      return enqueue_small(small, false, max_norm, scale, record, stream);
    // without a limit the norm is wanted for itself
    std::vector<NormArgs> norm = norm_launches(grads, numels, dtypes, n, std::isinf(max_norm) ? 0 : NORM_KEEP_BYTES);
    std::lock_guard<std::mutex> lock(api_mutex());
    return enqueue_norm(norm, max_norm, scale, record, workspace, stream);
  });
}

int muon_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                   const int* out_dtypes, int n, float max_norm, float scale, float* record, void* workspace,
                   hipStream_t stream) {
  return c_entry([&] {
    clear_error();
    int rc = validate_grad_clip(grads, outs, numels, dtypes, out_dtypes, n, max_norm, scale, record, workspace);
    if (rc) return rc;
    GradSmallArgs small;
    if (grad_small(grads, outs, numels, dtypes, out_dtypes, n, &small))
      return enqueue_small(small, true, max_norm, scale, record, stream);
    std::vector<ClipArgs> clip = clip_launches(grads, outs, numels, dtypes, out_dtypes, n);
    // in place the gradients are usually not read again
    bool in_place = true;
    for (const ClipArgs& a : clip) in_place = in_place && a.in_place;
    std::vector<NormArgs> norm = norm_launches(grads, numels, dtypes, n, in_place ? 0 : NORM_KEEP_BYTES);
    std::lock_guard<std::mutex> lock(api_mutex());
    if ((rc = enqueue_norm(norm, max_norm, scale, record, workspace, stream))) return rc;
    for (ClipArgs& a : clip) {
      a.record = record;
      if ((rc = timed(MUON_KERNEL_GRAD_CLIP, stream, [&] { return launch_grad_clip(a, stream); },
                      "gradient clip kernel launch")))
        return rc;
    }
    return MUON_OK;
  });
}

int muon_adamw_step_clip(float* const* params, const void* const* grads, const int* grad_dtypes,
                         float* const* exp_avg, float* const* exp_avg_sq, const int64_t* numels,
                         const float* weight_decay, int n, float lr, float beta1, float beta2, float eps,
                         int64_t step, const float* record, hipStream_t stream) {
  return c_entry([&] {
    clear_error();
    int rc = validate_adamw_clip(params, grads, grad_dtypes, exp_avg, exp_avg_sq, numels, weight_decay, n, lr, beta1,
                                 beta2, eps, step, record);
    if (rc) return rc;
    std::vector<AdamClipArgs> launches =
        adamw_clip_launches(params, grads, grad_dtypes, exp_avg, exp_avg_sq, numels, weight_decay, n);
    std::lock_guard<std::mutex> lock(api_mutex());
    for (AdamClipArgs& a : launches) {
      a.record = record;
      a.lr = lr;
      a.beta1 = beta1;
      a.beta2 = beta2;
      a.eps = eps;
      a.omb1 = (float)(1.0 - (double)beta1);
      a.omb2 = (float)(1.0 - (double)beta2);
      a.bc1 = (float)(1.0 - std::pow((double)beta1, (double)step));
      a.bc2 = (float)(1.0 - std::pow((double)beta2, (double)step));
      if ((rc = timed(MUON_KERNEL_ADAMW, stream, [&] { return launch_adamw_clip(a, stream); },
                      "adamw kernel launch")))
        return rc;
    }
    return MUON_OK;
  });
}

}  // extern "C"
