// Pieces of the C ABI's HIP side shared by its translation units: error
// text for HIP failures, stream-capture detection, the device addresses of a
// plan's tables and the launch sequence of one call.
#pragma once

#include <hip/hip_runtime.h>

#include <mutex>
#include <new>
#include <vector>

#include "muon_internal.h"
#include "plan_host.h"

namespace muon {

// Body of a C entry point: host allocation failure becomes MUON_ENOMEM, and no
// exception leaves the library.
template <typename F>
int c_entry(F&& body) noexcept {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return fail(MUON_ENOMEM, "host memory allocation failed");
  } catch (...) {
    return fail(MUON_EINVAL, "internal error");
  }
}

int fail_hip(hipError_t e, const char* what);
int capture_status(hipStream_t stream, bool* capturing);

// Timing of one kernel family (muon_timing_enable): its HIP events, as start
// and end pairs.
extern int g_time_kind;
extern std::vector<hipEvent_t> g_ev;
extern size_t g_ev_used;

// Launch wrapper: brackets the launch with events when its family is timed.
template <typename F>
int timed(int kind, hipStream_t stream, F&& launch, const char* what) {
  const bool on = (g_time_kind == kind);
  hipError_t e;
  if (on) {
    if (g_ev_used + 2 > g_ev.size()) {
      for (int k = 0; k < 2; ++k) {
        hipEvent_t ev;
        if ((e = hipEventCreate(&ev)) != hipSuccess) return fail_hip(e, "hipEventCreate");
        g_ev.push_back(ev);
      }
    }
    if ((e = hipEventRecord(g_ev[g_ev_used], stream)) != hipSuccess) return fail_hip(e, "hipEventRecord");
  }
  if ((e = launch()) != hipSuccess) return fail_hip(e, what);
  if (on) {
    if ((e = hipEventRecord(g_ev[g_ev_used + 1], stream)) != hipSuccess) return fail_hip(e, "hipEventRecord");
    g_ev_used += 2;
  }
  return MUON_OK;
}

// Serialises every entry point's use of the library's host state.
std::mutex& api_mutex();

// Device addresses of one lane's tables (a table block laid out as t says,
// over the workspace ws).
struct Tables {
  MatDesc* desc;
  int32_t* mats;
  int32_t* fin;
  EwItem *mom, *cast, *apply;
  GemmItem *gram, *poly, *upd;
  RedItem* red;
  float* gram_part;
  bool small;
  bool fused;
  int gram_tile, poly_tile, upd_tile, gram_bm;  // TileKind of each GEMM, Gram tile edge
  const LaneTables* t;
};
Tables tables_at(char* block, const PlanTables& t, int lane, char* ws);

// Pointer records into the descriptors at desc, PATCH_MAX per launch.
int patch_records(MatDesc* desc, const std::vector<PtrRecord>& recs, hipStream_t stream);

// The kernel sequence of one lane of a call (the caller holds api_mutex()).
// record: {norm, factor} on the device for a step on clipped gradients, or null.
int launch_sequence(int mode, const Tables& v, float lr, float beta, int ns_steps, const float* coeffs, int stride,
                    const float* record, hipStream_t stream);

}  // namespace muon
