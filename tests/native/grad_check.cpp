// Host check of the gradient calls' code (csrc/grad_host.cpp): refusals, and
// the launch tables walked the way the kernels walk them, so that every
// element of every tensor is covered exactly once and none outside.  Built
// with the host compiler under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_grad_host.py.  Prints "ok" and
// exits 0 when every check holds.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <limits>
#include <map>
#include <string>
#include <vector>

#include "grad_host.h"
#include "plan_host.h"

using namespace muon;

static int g_failures = 0;
#define CHECK(cond)                                                                   \
  do {                                                                                \
    if (!(cond)) {                                                                    \
      std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++g_failures;                                                                   \
    }                                                                                 \
  } while (0)

static bool refused(int rc, const char* text) {
  const bool ok = rc == MUON_EINVAL && std::string(last_error_text()).find(text) != std::string::npos;
  if (!ok) std::fprintf(stderr, "  rc %d, text \"%s\", expected \"%s\"\n", rc, last_error_text(), text);
  return ok;
}

// The kernels' search (grad_io.h): entries at or below the item, of the whole table.
static int find_tensor(const int32_t* start, int entries, int item) {
  int c = 0;
  for (int k = 0; k < entries; ++k) c += start[k] <= item;
  return c - 1;
}

static const int64_t kSizes[] = {0, 1, 3, 64, 4095, 4096, 4097, 8191, 8192, 8193, 12288, 40000, 1 << 20};

struct List {
  std::vector<int64_t> numel;
  std::vector<int> type, out_type;
  std::vector<const void*> g;
  std::vector<void*> out;
  std::vector<float*> p, u, v;
  std::vector<float> wd;
  int n() const { return (int)numel.size(); }
};

// Tensors far apart: addresses are only compared, never followed.
static List make_list(int n, int decays) {
  List l;
  uintptr_t a = (uintptr_t)1 << 32;
  auto next = [&] { a += (uintptr_t)1 << 26; return a + 4; };
  for (int i = 0; i < n; ++i) {
    l.numel.push_back(kSizes[(i * 7 + i / 13) % (sizeof kSizes / sizeof *kSizes)]);
    l.type.push_back(i % 3);
    l.out_type.push_back((i / 3) % 3);
    l.g.push_back((const void*)next());
    l.out.push_back((void*)next());
    l.p.push_back((float*)next());
    l.u.push_back((float*)next());
    l.v.push_back((float*)next());
    l.wd.push_back(0.01f * (float)(i % decays));
  }
  return l;
}

// Walks the items of one launch: seen[p] = elements covered of the tensor at p, in order.
template <typename Tail, typename Chunk>
static void walk(const int32_t* start, int entries, int n, int first, int stride, Tail tail, Chunk chunk,
                 std::map<int, std::vector<std::pair<int64_t, int>>>* seen) {
  for (int it = first; it < start[n]; it += stride) {
    const int t = find_tensor(start, entries, it);
    CHECK(t >= 0 && t < n && start[t] <= it && it < start[t + 1]);
    const int len = find_tensor(start, entries, it + 1) != t ? tail(t) : chunk(t);
    CHECK(len >= 1 && len <= chunk(t));
    (*seen)[t].push_back({(int64_t)(it - start[t]) * chunk(t), len});
  }
}

static int64_t covered(std::vector<std::pair<int64_t, int>> v) {
  // every piece once, back to back from 0
  std::map<int64_t, int> by(v.begin(), v.end());
  CHECK(by.size() == v.size());
  int64_t end = 0;
  for (auto& k : by) {
    CHECK(k.first == end);
    end += k.second;
  }
  return end;
}

static void check_norm(const List& l, int64_t keep) {
  const std::vector<NormArgs> a = norm_launches(l.g.data(), l.numel.data(), l.type.data(), l.n(), keep);
  CHECK(!a.empty() && a.front().first == 1 && a.back().last == 1);
  std::map<const void*, int64_t> got;
  int64_t items = 0, kept = 0;
  for (size_t k = 0; k < a.size(); ++k) {
    CHECK(a[k].keep_from >= 0 && a[k].keep_from <= a[k].start[a[k].n]);
    CHECK(k == 0 || a[k].keep_from == 0 || a[k - 1].keep_from == a[k - 1].start[a[k - 1].n]);  // the list's end
    items += a[k].start[a[k].n];
    kept += a[k].start[a[k].n] - a[k].keep_from;
    CHECK(a[k].first == (k == 0) && a[k].last == (k + 1 == a.size()));
    CHECK(a[k].blocks == a[0].blocks && a[k].blocks >= 1 && a[k].blocks <= NORM_MAX_BLOCKS);
    CHECK(a[k].n <= NORM_TENSORS && a[k].items == a[k].start[a[k].n]);
    std::map<int, std::vector<std::pair<int64_t, int>>> seen;
    for (int b = 0; b < a[k].blocks; ++b)
      walk(a[k].start, NORM_TENSORS + 1, a[k].n, b, a[k].blocks, [&](int t) { return (int)(a[k].tail[t] >> 2); },
           [&](int t) { return norm_chunk(a[k].tail[t] & 3); }, &seen);
    for (auto& s : seen) got[a[k].p[s.first]] += covered(s.second);
  }
  CHECK(kept == std::min(items, keep / NORM_CHUNK_BYTES));
  size_t full = 0;
  for (int i = 0; i < l.n(); ++i) {
    if (l.numel[i] == 0) continue;
    ++full;
    CHECK(got[l.g[i]] == l.numel[i]);
  }
  CHECK(got.size() == full);
}

static void check_clip(const List& l) {
  std::map<const void*, int64_t> got;
  for (const ClipArgs& a : clip_launches(l.g.data(), l.out.data(), l.numel.data(), l.type.data(), l.out_type.data(), l.n())) {
    CHECK(a.n >= 1 && a.n <= CLIP_TENSORS && a.items == a.start[a.n]);
    std::map<int, std::vector<std::pair<int64_t, int>>> seen;
    walk(a.start, CLIP_TENSORS + 1, a.n, 0, 1, [&](int t) { return (int)(a.tail[t] >> 4); }, [](int) { return CLIP_CHUNK; }, &seen);
    for (auto& s : seen) {
      got[a.out[s.first]] += covered(s.second);
      for (int i = 0; i < l.n(); ++i)
        if (l.out[i] == a.out[s.first])
          CHECK(l.g[i] == a.in[s.first] && (int)(a.tail[s.first] & 3) == l.type[i] &&
                (int)(a.tail[s.first] >> 2 & 3) == l.out_type[i]);
    }
  }
  for (int i = 0; i < l.n(); ++i) CHECK(got[l.out[i]] == l.numel[i]);
}

static void check_small(const List& l) {
  GradSmallArgs a, b;
  int64_t items = 0;
  for (int i = 0; i < l.n(); ++i) items += (l.numel[i] + norm_chunk(l.type[i]) - 1) / norm_chunk(l.type[i]);
  const bool small = grad_small(l.g.data(), l.out.data(), l.numel.data(), l.type.data(), l.out_type.data(), l.n(), &a);
  CHECK(small == (items <= NORM_SMALL_ITEMS));
  CHECK(small == grad_small(l.g.data(), nullptr, l.numel.data(), l.type.data(), nullptr, l.n(), &b));
  if (!small) return;
  CHECK(a.n <= NORM_SMALL_ITEMS && a.items == items && b.items == items && b.n == a.n);
  std::map<int, std::vector<std::pair<int64_t, int>>> seen;
  for (int wave = 0; wave < NORM_SMALL_ITEMS; ++wave)
    if (wave < a.items)
      walk(a.start, NORM_SMALL_ITEMS + 1, a.n, wave, NORM_SMALL_ITEMS, [&](int t) { return (int)(a.tail[t] >> 4); },
           [&](int t) { return norm_chunk(a.tail[t] & 3); }, &seen);
  std::map<const void*, int64_t> got;
  for (auto& s : seen) got[a.out[s.first]] += covered(s.second);
  for (int i = 0; i < l.n(); ++i) {
    CHECK(got[l.out[i]] == l.numel[i]);
    for (int t = 0; t < a.n; ++t)
      if (a.out[t] == l.out[i])
        CHECK(a.in[t] == l.g[i] && (int)(a.tail[t] & 3) == l.type[i] && (int)(a.tail[t] >> 2 & 3) == l.out_type[i]);
  }
}

static void check_adamw(const List& l, bool with_wd) {
  int64_t total = 0;
  for (int64_t m : l.numel) total += m;
  std::map<const void*, int64_t> got;
  for (const AdamClipArgs& a : adamw_clip_launches(l.p.data(), l.g.data(), l.type.data(), l.u.data(), l.v.data(),
                                                   l.numel.data(), with_wd ? l.wd.data() : nullptr, l.n())) {
    CHECK(a.n >= 1 && a.n <= ADAMC_TENSORS && a.items == a.start[a.n]);
    CHECK(a.chunk == (total >= ADAMC_LONG_MIN ? ADAMC_LONG_CHUNK : ADAMC_CHUNK));
    std::map<int, std::vector<std::pair<int64_t, int>>> seen;
    walk(a.start, ADAMC_TENSORS + 1, a.n, 0, 1, [&](int t) { return (int)(a.tail[t] >> 4); }, [&](int) { return a.chunk; }, &seen);
    for (auto& s : seen) {
      const int t = s.first;
      got[a.p[t]] += covered(s.second);
      for (int i = 0; i < l.n(); ++i)
        if (l.p[i] == a.p[t])
          CHECK(l.g[i] == a.g[t] && l.u[i] == a.u[t] && l.v[i] == a.v[t] && (int)(a.tail[t] & 3) == l.type[i] &&
                a.wd[a.tail[t] >> 2 & 3] == (with_wd ? l.wd[i] : 0.0f));
    }
  }
  for (int i = 0; i < l.n(); ++i) CHECK(got[l.p[i]] == l.numel[i]);
}

static void check_refusals() {
  const float inf = std::numeric_limits<float>::infinity(), nan = std::numeric_limits<float>::quiet_NaN();
  float* const rec = (float*)0x900000;
  void* const ws = (void*)0xa00000;
  const void* g[2] = {(void*)0x100000, (void*)0x200000};
  void* o[2] = {(void*)0x300000, (void*)0x400000};
  float *p[2] = {(float*)0x300000, (float*)0x400000}, *u[2] = {(float*)0x500000, (float*)0x600000},
        *v[2] = {(float*)0x700000, (float*)0x800000};
  int64_t numel[2] = {100, 200};
  int t32[2] = {MUON_FP32, MUON_FP32}, t16[2] = {MUON_BF16, MUON_FP16}, bad[2] = {MUON_FP32, 3};

  // the norm
  CHECK(validate_grad_norm(g, numel, t16, 2, inf, 1.0f, rec, ws) == MUON_OK);
  CHECK(validate_grad_norm(nullptr, nullptr, nullptr, 0, 1.0f, 1.0f, rec, ws) == MUON_OK);
  CHECK(refused(validate_grad_norm(g, numel, t32, -1, 1.0f, 1.0f, rec, ws), "n = -1"));
  CHECK(refused(validate_grad_norm(g, numel, t32, MUON_GRAD_MAX_TENSORS + 1, 1.0f, 1.0f, rec, ws), "outside"));
  CHECK(refused(validate_grad_norm(nullptr, numel, t32, 2, 1.0f, 1.0f, rec, ws), "NULL"));
  CHECK(refused(validate_grad_norm(g, numel, bad, 2, 1.0f, 1.0f, rec, ws), "dtypes[1] = 3"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, nan, 1.0f, rec, ws), "max_norm"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, -1.0f, 1.0f, rec, ws), "max_norm"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 0.0f, rec, ws), "scale"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, inf, rec, ws), "scale"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 1.0f, nullptr, ws), "record is NULL"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 1.0f, (float*)0x900002, ws), "record is not"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 1.0f, rec, nullptr), "workspace is NULL"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 1.0f, rec, (char*)ws + 8), "workspace is not"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 1.0f, rec, (char*)rec - 16), "record overlaps workspace"));
  CHECK(refused(validate_grad_norm(g, numel, t32, 2, 1.0f, 1.0f, (float*)0x100004, ws), "overlaps grads[0]"));
  {
    const void* q[2] = {g[0], (void*)0x200002};
    CHECK(refused(validate_grad_norm(q, numel, t32, 2, 1.0f, 1.0f, rec, ws), "grads[1] is not 4-byte"));
    CHECK(validate_grad_norm(q, numel, t16, 2, 1.0f, 1.0f, rec, ws) == MUON_OK);  // 16-bit elements: 2-byte aligned
    const void* z[2] = {g[0], nullptr};
    CHECK(refused(validate_grad_norm(z, numel, t32, 2, 1.0f, 1.0f, rec, ws), "grads[1] is NULL"));
    int64_t m[2] = {100, 0};
    CHECK(validate_grad_norm(z, m, t32, 2, 1.0f, 1.0f, rec, ws) == MUON_OK);
    m[1] = -1;
    CHECK(refused(validate_grad_norm(g, m, t32, 2, 1.0f, 1.0f, rec, ws), "negative"));
    m[1] = GRAD_MAX_NUMEL + 1;
    CHECK(refused(validate_grad_norm(g, m, t32, 2, 1.0f, 1.0f, rec, ws), "too large"));
    const void* same[2] = {g[0], g[0]};
    CHECK(validate_grad_norm(same, numel, t32, 2, 1.0f, 1.0f, rec, ws) == MUON_OK);  // read only
  }
  // clipping
  CHECK(validate_grad_clip(g, o, numel, t16, t32, 2, 1.0f, 1.0f, rec, ws) == MUON_OK);
  CHECK(refused(validate_grad_clip(g, o, numel, t16, bad, 2, 1.0f, 1.0f, rec, ws), "out_dtypes[1] = 3"));
  {
    void* in_place[2] = {(void*)g[0], (void*)g[1]};
    CHECK(validate_grad_clip(g, in_place, numel, t16, t16, 2, 1.0f, 1.0f, rec, ws) == MUON_OK);
    CHECK(refused(validate_grad_clip(g, in_place, numel, t16, t32, 2, 1.0f, 1.0f, rec, ws), "of another type"));
    const void* same[2] = {g[0], g[0]};
    void* twice[2] = {(void*)g[0], (void*)g[0]};
    CHECK(refused(validate_grad_clip(same, twice, numel, t32, t32, 2, 1.0f, 1.0f, rec, ws), "overlaps outs"));
    CHECK(validate_grad_clip(same, o, numel, t32, t32, 2, 1.0f, 1.0f, rec, ws) == MUON_OK);
    // an out inside a long gradient that starts before a shorter one
    const void* nest[2] = {(void*)0x100000, (void*)0x100010};
    void* into[2] = {(void*)0x300000, (void*)0x100100};
    CHECK(refused(validate_grad_clip(nest, into, numel, t32, t32, 2, 1.0f, 1.0f, rec, ws), "outs[1] overlaps grads"));
    void* cross[2] = {(void*)g[1], o[1]};
    CHECK(refused(validate_grad_clip(g, cross, numel, t32, t32, 2, 1.0f, 1.0f, rec, ws), "overlaps"));
    void* at_record[2] = {o[0], (char*)rec - 8};
    CHECK(refused(validate_grad_clip(g, at_record, numel, t32, t32, 2, 1.0f, 1.0f, rec, ws), "record overlaps outs[1]"));
    void* null[2] = {o[0], nullptr};
    CHECK(refused(validate_grad_clip(g, null, numel, t32, t32, 2, 1.0f, 1.0f, rec, ws), "outs[1] is NULL"));
  }
  // AdamW
  auto adamw = [&](const void* const* gr, const int* ty, float* const* uu, const float* wd, float b1, int64_t step,
                   const float* r) {
    return validate_adamw_clip(p, gr, ty, uu, v, numel, wd, 2, 1e-3f, b1, 0.999f, 1e-8f, step, r);
  };
  const float wd_ok[2] = {0.0f, 0.1f}, wd_bad[2] = {0.0f, -0.1f};
  CHECK(adamw(g, t16, u, wd_ok, 0.9f, 1, rec) == MUON_OK);
  CHECK(adamw(g, t32, u, nullptr, 0.9f, 1, nullptr) == MUON_OK);
  CHECK(refused(adamw(g, bad, u, wd_ok, 0.9f, 1, rec), "grad_dtypes[1]"));
  CHECK(refused(adamw(g, t32, u, wd_bad, 0.9f, 1, rec), "weight_decay[1]"));
  CHECK(refused(adamw(g, t32, u, wd_ok, 1.0f, 1, rec), "beta1"));
  CHECK(refused(adamw(g, t32, u, wd_ok, 0.9f, 0, rec), "step"));
  CHECK(refused(adamw(g, t32, u, wd_ok, 0.9f, 1, (float*)0x900001), "record is not"));
  CHECK(refused(adamw(g, t32, u, wd_ok, 0.9f, 1, u[1]), "overlaps"));
  CHECK(refused(adamw(g, t32, p, wd_ok, 0.9f, 1, rec), "overlaps"));
  CHECK(refused(validate_adamw_clip(p, g, nullptr, u, v, numel, nullptr, 2, 1e-3f, 0.9f, 0.999f, 1e-8f, 1, rec), "NULL"));
  // the record of a Muon step
  const muon_shape_t shapes[2] = {{10, 10}, {10, 20}};
  CHECK(validate_step_record(p, u, nullptr, shapes, 2, rec) == MUON_OK);
  CHECK(refused(validate_step_record(p, u, nullptr, shapes, 2, (float*)0x900002), "record is not"));
  CHECK(refused(validate_step_record(p, u, nullptr, shapes, 2, u[0] + 99), "overlaps"));
  uint16_t* upd[2] = {nullptr, (uint16_t*)rec};
  CHECK(refused(validate_step_record(p, u, upd, shapes, 2, rec), "overlaps"));
}

int main() {
  for (int n : {0, 1, 2, 3, 4, 5, 6, 7, 8, 99, 100, 101, 167, 168, 169, 251, 252, 253, 600}) {
    for (int decays : {1, 4, 5, 9}) {
      const List l = make_list(n, decays);
      if (decays == 1) {
        for (int64_t keep : {(int64_t)0, (int64_t)1 << 20, NORM_KEEP_BYTES}) check_norm(l, keep);
        check_clip(l);
        check_small(l);
      }
      check_adamw(l, true);
      check_adamw(l, false);
    }
  }
  // as many items as the small call takes, and one more
  for (int n : {15, 16, 17}) {
    List l = make_list(n, 1);
    for (int i = 0; i < n; ++i) l.numel[i] = i % 2 ? 1 : norm_chunk(l.type[i]);
    check_small(l);
  }
  // a call long enough for the long chunks
  {
    List l = make_list(130, 3);
    for (int i = 0; i < 130; ++i) l.numel[i] += (int64_t)1 << 20;
    check_adamw(l, true);
    check_norm(l, NORM_KEEP_BYTES);
  }
  // two decays in one launch; nine need three launches, in whatever order they come
  {
    List l = make_list(60, 5);
    for (int i = 0; i < 60; ++i) l.numel[i] = 64;
    for (int i = 0; i < 60; ++i) l.wd[i] = i < 30 ? 0.0f : 0.1f;
    CHECK(adamw_clip_launches(l.p.data(), l.g.data(), l.type.data(), l.u.data(), l.v.data(), l.numel.data(),
                              l.wd.data(), 60).size() == 1);
    for (int i = 0; i < 60; ++i) l.wd[i] = 0.01f * (float)(i % 9);  // in turn: taken decay by decay
    CHECK(adamw_clip_launches(l.p.data(), l.g.data(), l.type.data(), l.u.data(), l.v.data(), l.numel.data(),
                              l.wd.data(), 60).size() == 3);
  }
  // a list whose items pass the grid limit is cut, and offsets pass 32 bits
  {
    std::vector<int64_t> numel(20, GRAD_MAX_NUMEL);
    std::vector<int> type(20, MUON_BF16);
    std::vector<const void*> g(20);
    std::vector<void*> o(20);
    for (int i = 0; i < 20; ++i) g[i] = o[i] = (void*)((uintptr_t)(i + 1) << 44);
    int64_t items = 0;
    for (const NormArgs& a : norm_launches(g.data(), numel.data(), type.data(), 20, NORM_KEEP_BYTES)) {
      CHECK(a.start[a.n] <= MAX_LAUNCH_ITEMS && a.start[a.n] >= 0);
      items += a.start[a.n];
    }
    CHECK(items == 20 * (GRAD_MAX_NUMEL / norm_chunk(MUON_BF16)));
    items = 0;
    for (const ClipArgs& a : clip_launches(g.data(), o.data(), numel.data(), type.data(), type.data(), 20)) {
      CHECK(a.items <= MAX_LAUNCH_ITEMS);
      items += a.items;
    }
    CHECK(items == 20 * (GRAD_MAX_NUMEL / CLIP_CHUNK));
  }
  check_refusals();
  if (g_failures) return 1;
  std::printf("ok\n");
  return 0;
}
