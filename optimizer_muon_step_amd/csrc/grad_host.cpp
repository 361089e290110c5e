// Validation and launch tables of the gradient-norm, clipping and
// clipped-AdamW entry points.  No GPU calls.
#include "grad_host.h"

#include <algorithm>
#include <cmath>
#include <string>

#include "plan_host.h"

namespace muon {

static_assert(GRAD_FP32 == MUON_FP32 && GRAD_BF16 == MUON_BF16 && GRAD_FP16 == MUON_FP16, "type codes");
static_assert(sizeof(NormWorkspace) <= MUON_GRAD_WORKSPACE_BYTES, "workspace size");

namespace {

struct Span {
  uintptr_t lo, hi;
  bool written;
  int tensor;  // -1: not one of a list
  const char* what;
};

std::string name_of(const Span& s) {
  return s.tensor < 0 ? std::string(s.what) : std::string(s.what) + "[" + std::to_string(s.tensor) + "]";
}

bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// No written array may overlap another one; read arrays may share memory.
int check_spans(std::vector<Span>& v) {
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  const Span *any = nullptr, *wr = nullptr;  // of the spans so far, those reaching furthest
  for (const Span& s : v) {
    const Span* other = s.written ? any : wr;
    if (other && s.lo < other->hi)
      return fail(MUON_EINVAL, "%s overlaps %s", name_of(s).c_str(), name_of(*other).c_str());
    if (!any || s.hi > any->hi) any = &s;
    if (s.written && (!wr || s.hi > wr->hi)) wr = &s;
  }
  return MUON_OK;
}

int check_count(int n) {
  if (n < 0 || n > MUON_GRAD_MAX_TENSORS) return fail(MUON_EINVAL, "n = %d outside [0, %d]", n, MUON_GRAD_MAX_TENSORS);
  return MUON_OK;
}

int check_numel(const int64_t* numels, int i) {
  if (numels[i] < 0) return fail(MUON_EINVAL, "numels[%d] = %lld is negative", i, (long long)numels[i]);
  if (numels[i] > GRAD_MAX_NUMEL) return fail(MUON_EINVAL, "numels[%d] = %lld is too large", i, (long long)numels[i]);
  return MUON_OK;
}

int check_type(const int* types, int i, const char* what) {
  if (types[i] < MUON_FP32 || types[i] > MUON_FP16)
    return fail(MUON_EINVAL, "%s[%d] = %d is no element type (MUON_FP32, MUON_BF16, MUON_FP16)", what, i, types[i]);
  return MUON_OK;
}

int check_ptr(const void* p, int type, int i, const char* what) {
  if (!p) return fail(MUON_EINVAL, "%s[%d] is NULL", what, i);
  if ((uintptr_t)p % grad_type_bytes(type))
    return fail(MUON_EINVAL, "%s[%d] is not %d-byte aligned", what, i, grad_type_bytes(type));
  return MUON_OK;
}

Span span_of(const void* p, size_t bytes, bool written, int i, const char* what) {
  return {(uintptr_t)p, (uintptr_t)p + bytes, written, i, what};
}

int check_clip_scalars(float max_norm, float scale, const float* record, const void* workspace) {
  if (std::isnan(max_norm) || max_norm < 0.0f) return fail(MUON_EINVAL, "max_norm = %g is not >= 0", (double)max_norm);
  if (!std::isfinite(scale) || scale <= 0.0f) return fail(MUON_EINVAL, "scale = %g is not finite and > 0", (double)scale);
  if (!record) return fail(MUON_EINVAL, "record is NULL");
  if ((uintptr_t)record % 4) return fail(MUON_EINVAL, "record is not 4-byte aligned");
  if (!workspace) return fail(MUON_EINVAL, "workspace is NULL");
  if ((uintptr_t)workspace % 16) return fail(MUON_EINVAL, "workspace is not 16-byte aligned");
  return MUON_OK;
}

// Items of one tensor and the element count of its last one.
struct Cut {
  int64_t items;
  uint32_t last;
};
Cut cut_of(int64_t numel, int chunk) {
  const int64_t items = (numel + chunk - 1) / chunk;
  return {items, (uint32_t)(numel - (items - 1) * chunk)};
}

template <typename Args>
void fill_unused(Args& a) {
  std::fill(a.start + a.n + 1, a.start + sizeof a.start / sizeof *a.start, START_UNUSED);
}

}  // namespace

int validate_grad_norm(const void* const* grads, const int64_t* numels, const int* types, int n, float max_norm,
                       float scale, const float* record, const void* workspace) {
  int rc = check_count(n);
  if (rc) return rc;
  if (n > 0 && (!grads || !numels || !types))
    return fail(MUON_EINVAL, "grads, numels and dtypes arrays must not be NULL");
  if ((rc = check_clip_scalars(max_norm, scale, record, workspace))) return rc;
  // only these two are written: no need to put every gradient in order
  const Span written[2] = {span_of(record, MUON_CLIP_RECORD_FLOATS * sizeof(float), true, -1, "record"),
                           span_of(workspace, MUON_GRAD_WORKSPACE_BYTES, true, -1, "workspace")};
  if (overlap(written[0], written[1])) return fail(MUON_EINVAL, "record overlaps workspace");
  for (int i = 0; i < n; ++i) {
    if ((rc = check_numel(numels, i)) || (rc = check_type(types, i, "dtypes"))) return rc;
    if (numels[i] == 0) continue;
    if ((rc = check_ptr(grads[i], types[i], i, "grads"))) return rc;
    const Span g = span_of(grads[i], (size_t)numels[i] * grad_type_bytes(types[i]), false, i, "grads");
    for (const Span& w : written)
      if (overlap(w, g)) return fail(MUON_EINVAL, "%s overlaps %s", w.what, name_of(g).c_str());
  }
  return MUON_OK;
}

int validate_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* types,
                       const int* out_types, int n, float max_norm, float scale, const float* record,
                       const void* workspace) {
  int rc = check_count(n);
  if (rc) return rc;
  if (n > 0 && (!grads || !outs || !numels || !types || !out_types))
    return fail(MUON_EINVAL, "grads, outs, numels, dtypes and out_dtypes arrays must not be NULL");
  if ((rc = check_clip_scalars(max_norm, scale, record, workspace))) return rc;
  std::vector<Span> v;
  v.reserve(2 * (size_t)n + 2);
  v.push_back(span_of(record, MUON_CLIP_RECORD_FLOATS * sizeof(float), true, -1, "record"));
  v.push_back(span_of(workspace, MUON_GRAD_WORKSPACE_BYTES, true, -1, "workspace"));
  for (int i = 0; i < n; ++i) {
    if ((rc = check_numel(numels, i)) || (rc = check_type(types, i, "dtypes")) ||
        (rc = check_type(out_types, i, "out_dtypes")))
      return rc;
    if (numels[i] == 0) continue;
    if ((rc = check_ptr(grads[i], types[i], i, "grads")) || (rc = check_ptr(outs[i], out_types[i], i, "outs")))
      return rc;
    const bool in_place = grads[i] == outs[i];
    if (in_place && types[i] != out_types[i])
      return fail(MUON_EINVAL, "outs[%d] is grads[%d], but of another type", i, i);
    v.push_back(span_of(outs[i], (size_t)numels[i] * grad_type_bytes(out_types[i]), true, i, "outs"));
    if (!in_place) v.push_back(span_of(grads[i], (size_t)numels[i] * grad_type_bytes(types[i]), false, i, "grads"));
  }
  return check_spans(v);
}

int validate_adamw_clip(float* const* params, const void* const* grads, const int* types, float* const* u,
                        float* const* v, const int64_t* numels, const float* wd, int n, float lr, float beta1,
                        float beta2, float eps, int64_t step, const float* record) {
  int rc = check_count(n);
  if (rc) return rc;
  if (n > 0 && (!params || !grads || !types || !u || !v || !numels))
    return fail(MUON_EINVAL, "params, grads, grad_dtypes, exp_avg, exp_avg_sq and numels arrays must not be NULL");
  if ((rc = check_adamw_scalars(lr, beta1, beta2, eps, step))) return rc;
  if ((uintptr_t)record % 4) return fail(MUON_EINVAL, "record is not 4-byte aligned");
  std::vector<Span> s;
  s.reserve(4 * (size_t)n + 1);
  if (record) s.push_back(span_of(record, MUON_CLIP_RECORD_FLOATS * sizeof(float), false, -1, "record"));
  for (int i = 0; i < n; ++i) {
    if ((rc = check_numel(numels, i)) || (rc = check_type(types, i, "grad_dtypes"))) return rc;
    if (wd && (!std::isfinite(wd[i]) || wd[i] < 0.0f))
      return fail(MUON_EINVAL, "weight_decay[%d] = %g is not finite and >= 0", i, (double)wd[i]);
    if (numels[i] == 0) continue;
    const size_t fb = (size_t)numels[i] * sizeof(float);
    if ((rc = check_ptr(params[i], GRAD_FP32, i, "params")) || (rc = check_ptr(grads[i], types[i], i, "grads")) ||
        (rc = check_ptr(u[i], GRAD_FP32, i, "exp_avg")) || (rc = check_ptr(v[i], GRAD_FP32, i, "exp_avg_sq")))
      return rc;
    s.push_back(span_of(params[i], fb, true, i, "params"));
    s.push_back(span_of(u[i], fb, true, i, "exp_avg"));
    s.push_back(span_of(v[i], fb, true, i, "exp_avg_sq"));
    s.push_back(span_of(grads[i], (size_t)numels[i] * grad_type_bytes(types[i]), false, i, "grads"));
  }
  return check_spans(s);
}

int validate_step_record(float* const* params, float* const* moms, uint16_t* const* upd, const muon_shape_t* shapes,
                         int n, const float* record) {
  if ((uintptr_t)record % 4) return fail(MUON_EINVAL, "record is not 4-byte aligned");
  std::vector<Span> s;
  s.reserve(3 * (size_t)n + 1);
  s.push_back(span_of(record, MUON_CLIP_RECORD_FLOATS * sizeof(float), false, -1, "record"));
  for (int i = 0; i < n; ++i) {
    const size_t numel = (size_t)shapes[i].rows * shapes[i].cols;
    s.push_back(span_of(params[i], numel * sizeof(float), true, i, "params"));
    s.push_back(span_of(moms[i], numel * sizeof(float), true, i, "momentum"));
    if (upd && upd[i]) s.push_back(span_of(upd[i], numel * sizeof(uint16_t), true, i, "updates"));
  }
  return check_spans(s);
}

bool grad_small(const void* const* grads, void* const* outs, const int64_t* numels, const int* types,
                const int* out_types, int n, GradSmallArgs* out) {
  GradSmallArgs a{};
  for (int i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const Cut c = cut_of(numels[i], norm_chunk(types[i]));
    if (a.items + c.items > NORM_SMALL_ITEMS) return false;  // then there are no more tensors than items either
    a.tail[a.n] = c.last << 4 | (uint32_t)(outs ? out_types[i] : 0) << 2 | (uint32_t)types[i];
    a.in[a.n] = grads[i];
    a.out[a.n] = outs ? outs[i] : nullptr;
    a.items += (int32_t)c.items;
    a.start[++a.n] = a.items;
  }
  fill_unused(a);
  *out = a;
  return true;
}

std::vector<NormArgs> norm_launches(const void* const* grads, const int64_t* numels, const int* types, int n,
                                    int64_t keep_bytes) {
  std::vector<NormArgs> out(1, NormArgs{});
  for (int i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const Cut c = cut_of(numels[i], norm_chunk(types[i]));
    NormArgs* a = &out.back();
    if (a->n == NORM_TENSORS || (a->n > 0 && a->items + c.items > MAX_LAUNCH_ITEMS)) {
      out.push_back(NormArgs{});
      a = &out.back();
    }
    a->tail[a->n] = c.last << 2 | (uint32_t)types[i];
    a->p[a->n] = grads[i];
    a->items += (int32_t)c.items;
    a->start[++a->n] = a->items;
  }
  for (NormArgs& a : out) fill_unused(a);
  out.front().first = 1;
  out.back().last = 1;
  int64_t left = keep_bytes;
  for (auto a = out.rbegin(); a != out.rend(); ++a) {
    const int64_t items = std::min<int64_t>(a->items, left / NORM_CHUNK_BYTES);
    a->keep_from = a->items - (int32_t)items;
    left -= items * NORM_CHUNK_BYTES;
  }
  int32_t most = 1;
  for (const NormArgs& a : out) most = std::max(most, a.items);
  for (NormArgs& a : out) a.blocks = std::min(most, (int32_t)NORM_MAX_BLOCKS);
  return out;
}

std::vector<ClipArgs> clip_launches(const void* const* grads, void* const* outs, const int64_t* numels,
                                    const int* types, const int* out_types, int n) {
  std::vector<ClipArgs> out;
  for (int i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const Cut c = cut_of(numels[i], CLIP_CHUNK);
    if (out.empty() || out.back().n == CLIP_TENSORS || out.back().items + c.items > MAX_LAUNCH_ITEMS) {
      out.push_back(ClipArgs{});
      out.back().in_place = 1;
    }
    ClipArgs& a = out.back();
    a.in_place &= grads[i] == outs[i];
    a.tail[a.n] = c.last << 4 | (uint32_t)out_types[i] << 2 | (uint32_t)types[i];
    a.in[a.n] = grads[i];
    a.out[a.n] = outs[i];
    a.items += (int32_t)c.items;
    a.start[++a.n] = a.items;
  }
  for (auto& a : out) fill_unused(a);
  return out;
}

std::vector<AdamClipArgs> adamw_clip_launches(float* const* params, const void* const* grads, const int* types,
                                              float* const* u, float* const* v, const int64_t* numels,
                                              const float* wd, int n) {
  std::vector<AdamClipArgs> out;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += numels[i];
  const int chunk = total >= ADAMC_LONG_MIN ? ADAMC_LONG_CHUNK : ADAMC_CHUNK;
  // A launch holds ADAMC_DECAYS distinct decays: with more of them the tensors
  // are taken decay by decay (their order changes no result).
  std::vector<int> order;
  std::vector<float> seen;
  for (int i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    order.push_back(i);
    const float lambda = wd ? wd[i] : 0.0f;
    if (seen.size() <= (size_t)ADAMC_DECAYS && std::find(seen.begin(), seen.end(), lambda) == seen.end())
      seen.push_back(lambda);
  }
  if (seen.size() > (size_t)ADAMC_DECAYS)
    std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return wd[x] < wd[y]; });
  int decays = 0;  // distinct ones of the last launch so far
  for (int i : order) {
    const Cut c = cut_of(numels[i], chunk);
    const float lambda = wd ? wd[i] : 0.0f;
    int k = 0;
    if (!out.empty())
      while (k < decays && out.back().wd[k] != lambda) ++k;
    if (out.empty() || out.back().n == ADAMC_TENSORS || k == ADAMC_DECAYS ||
        out.back().items + c.items > MAX_LAUNCH_ITEMS) {
      out.push_back(AdamClipArgs{});
      out.back().chunk = chunk;
      k = decays = 0;
    }
    AdamClipArgs& a = out.back();
    if (k == decays) a.wd[decays++] = lambda;
    a.tail[a.n] = c.last << 4 | (uint32_t)k << 2 | (uint32_t)types[i];
    a.p[a.n] = params[i];
    a.g[a.n] = grads[i];
    a.u[a.n] = u[i];
    a.v[a.n] = v[i];
    a.items += (int32_t)c.items;
    a.start[++a.n] = a.items;
  }
  for (auto& a : out) fill_unused(a);
  return out;
}

}  // namespace muon
