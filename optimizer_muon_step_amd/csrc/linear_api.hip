// C ABI of the hidden layers' products and of dropout: each call validates on
// the host and enqueues its launches; everything travels as kernel arguments,
// so nothing is cached or allocated on the device.
#include <hip/hip_runtime.h>

#include <mutex>

#include "../../include/muon.h"
#include "api_internal.h"
#include "linear_host.h"
#include "muon_internal.h"

namespace muon {
namespace {

int enqueue_pack(const LinPlan& p, int kind, hipStream_t stream) {
  if (p.pack.n == 0) return MUON_OK;
  return timed(kind, stream, [&] { return launch_linear_pack(p.pack, stream); }, "operand copy kernel launch");
}

int enqueue_layer(const muon_linear_t* l, bool backward, void* workspace, size_t bytes, hipStream_t stream) {
  clear_error();
  LinPlan p;
  int rc = plan_linear(l, backward, workspace, bytes, &p);
  if (rc || p.empty) return rc;
  std::lock_guard<std::mutex> lock(api_mutex());
  if ((rc = enqueue_pack(p, MUON_KERNEL_LINEAR, stream))) return rc;
  rc = timed(MUON_KERNEL_LINEAR, stream, [&] { return launch_linear(p.gemm, p.type, p.b_kmajor, p.b_wide, p.tile, stream); },
             "layer product kernel launch");
  if (rc || !p.finish) return rc;
  return timed(MUON_KERNEL_LINEAR, stream, [&] { return launch_linear_join(p.join, p.type, stream); },
               "layer product kernel launch");
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t muon_linear_workspace_bytes(const muon_linear_t* l, int backward) {
  size_t bytes = 0;
  c_entry([&] {
    clear_error();
    return linear_workspace(l, backward != 0, &bytes);
  });
  return bytes;
}

int muon_linear(const muon_linear_t* l, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return c_entry([&] { return enqueue_layer(l, false, workspace, workspace_bytes, stream); });
}

int muon_linear_dx(const muon_linear_t* l, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return c_entry([&] { return enqueue_layer(l, true, workspace, workspace_bytes, stream); });
}

size_t muon_linear_dw_workspace_bytes(const muon_linear_dw_t* l) {
  size_t bytes = 0;
  c_entry([&] {
    clear_error();
    return linear_dw_workspace(l, &bytes);
  });
  return bytes;
}

int muon_linear_dw(const muon_linear_dw_t* l, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return c_entry([&] {
    clear_error();
    LinPlan p;
    int rc = plan_linear_dw(l, workspace, workspace_bytes, &p);
    if (rc || p.empty) return rc;
    std::lock_guard<std::mutex> lock(api_mutex());
    if ((rc = enqueue_pack(p, MUON_KERNEL_LINEAR_DW, stream))) return rc;
    rc = timed(MUON_KERNEL_LINEAR_DW, stream, [&] { return launch_linear_dw(p.gemm, p.type, p.tile, stream); },
               "weight gradient kernel launch");
    if (rc || !p.finish) return rc;
    return timed(MUON_KERNEL_LINEAR_DW, stream, [&] { return launch_linear_finish(p.fin, stream); },
                 "weight gradient kernel launch");
  });
}

int muon_dropout(const muon_dropout_t* d, hipStream_t stream) {
  return c_entry([&] {
    clear_error();
    DropArgs a;
    int64_t blocks;
    const int rc = plan_dropout(d, &a, &blocks);
    if (rc || blocks == 0) return rc;
    std::lock_guard<std::mutex> lock(api_mutex());
    return timed(MUON_KERNEL_DROPOUT, stream, [&] { return launch_dropout(a, blocks, stream); }, "dropout kernel launch");
  });
}

}  // extern "C"
