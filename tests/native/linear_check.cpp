// Host check of the layer products' and dropout's code (csrc/linear_host.cpp):
// refusals, what shares memory and what does not, and the launch arguments
// against the sizes they stand for.  Built with the host compiler under
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_linear_host.py.
// Prints "ok" and exits 0 when every check holds.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <limits>
#include <set>
#include <string>

#include "linear_host.h"
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

static bool said(int rc, int want, const char* text) {
  const bool ok = rc == want && std::string(last_error_text()).find(text) != std::string::npos;
  if (!ok) std::fprintf(stderr, "  rc %d, text \"%s\", expected \"%s\"\n", rc, last_error_text(), text);
  return ok;
}

// Addresses are only compared, never followed.
static void* at(uint64_t gib, uint64_t bytes = 0) { return (void*)(uintptr_t)((gib << 30) + bytes); }

static muon_linear_t layer(int64_t m, int64_t k, int64_t n, bool backward = false, int w_t = 0) {
  muon_linear_t l = {};
  l.m = m;
  l.k = k;
  l.n = n;
  l.x = at(64);
  l.w = at(128);
  l.y = at(192);
  l.ldx = backward ? n : k;
  l.ldy = backward ? k : n;
  l.ldw = w_t ? k : n;
  l.w_transposed = w_t;
  l.x_type = l.w_type = l.y_type = l.bias_type = MUON_BF16;
  return l;
}

static int run(const muon_linear_t& l, bool backward = false, LinPlan* out = nullptr) {
  LinPlan p;
  size_t bytes = 0;
  linear_workspace(&l, backward, &bytes);
  return plan_linear(&l, backward, at(512), bytes, out ? out : &p);
}

// The launch covers the product and no more than a tile beyond it.
static void check_gemm(const LinPlan& p, int64_t m, int64_t n, int64_t k) {
  const LinGemmArgs& g = p.gemm;
  const LinTileSize t = kLinTile[p.tile];
  CHECK(g.m == m && g.n == n && g.k == k);
  CHECK((int64_t)g.tiles_m * t.bm >= m && (int64_t)(g.tiles_m - 1) * t.bm < m);
  CHECK((int64_t)g.tiles_n * t.bn >= n && (int64_t)(g.tiles_n - 1) * t.bn < n);
  CHECK((int64_t)g.slices * t.bk >= k && (int64_t)(g.slices - 1) * t.bk < k);
  CHECK(g.splits >= 1 && (int64_t)g.splits * g.per_split >= g.slices && (g.splits - 1) * g.per_split < std::max(1, g.slices));
  for (const LinOperand* o : {&g.a, &g.b}) {
    if (k == 0 || p.tile == LIN_TILE_64_ANY) continue;
    CHECK((uintptr_t)o->p % 16 == 0 && o->ld % 16 == 0 && o->ld < ((int64_t)1 << 24) && o->bytes % 16 == 0);
    CHECK(255 * o->ld + 128 < 0x7ffffff0);  // a tile's offsets
  }
}

static void check_layers() {
  std::set<int> tiles;
  for (int64_t m : {1, 2, 31, 64, 100, 1000, 4097, 16384, 100000})
    for (int64_t k : {1, 7, 8, 72, 768, 1001, 4096})
      for (int64_t n : {1, 8, 40, 771, 2304, 6400})
        for (int v = 0; v < 8; ++v) {
          const bool backward = v & 1;
          muon_linear_t l = layer(m, k, n, backward, (v >> 1) & 1);
          if (v & 4) l.w_type = MUON_FP32;
          const int64_t in = backward ? n : k, out = backward ? k : n;
          LinPlan p;
          CHECK(run(l, backward, &p) == MUON_OK);
          check_gemm(p, m, out, in);
          tiles.insert(p.tile);
          const bool x_copied = in % 8 != 0, w_copied = (v & 4) || (l.w_transposed ? k : n) % 8 != 0;
          if (p.tile == LIN_TILE_64_ANY) {
            CHECK((x_copied || w_copied) && in >= 8 && (l.w_transposed ? k : n) >= 8 && p.b_wide == ((v & 4) != 0));
            CHECK(p.pack.n == 0 && p.gemm.a.p == l.x && p.gemm.b.p == l.w);
            CHECK(p.gemm.a.ld == l.ldx * 2 && p.gemm.b.ld == l.ldw * (v & 4 ? 4 : 2));
          } else {
            CHECK(p.pack.n == x_copied + w_copied && !p.b_wide);
            CHECK((p.gemm.a.p == l.x) == !x_copied && (p.gemm.b.p == l.w) == !w_copied);
          }
          // copies lie in the workspace, apart from one another
          uintptr_t end = (uintptr_t)at(512);
          for (int i = 0; i < p.pack.n; ++i) {
            const LinPack& c = p.pack.job[i];
            CHECK((uintptr_t)c.dst >= end && c.dst_ld >= c.cols && c.dst_ld % 8 == 0);
            end = (uintptr_t)c.dst + (size_t)(c.rows * c.dst_ld * 2);
          }
          CHECK(end <= (uintptr_t)at(512) + p.workspace && p.workspace % 256 == 0);
          CHECK(p.finish == (p.gemm.splits > 1));
          if (p.finish) {  // the sums of the splits lie behind the copies
            const LinTileSize t = kLinTile[p.tile];
            const LinJoinArgs& j = p.join;
            CHECK(j.m == m && j.n == out && j.splits == p.gemm.splits && j.part == p.gemm.part && (uintptr_t)j.part >= end);
            CHECK(j.part_ld == (int64_t)p.gemm.tiles_n * t.bn && j.part_stride == j.part_ld * p.gemm.tiles_m * t.bm);
            CHECK((const char*)(j.part + j.part_stride * j.splits) <= (const char*)at(512) + p.workspace);
            CHECK(j.e.y == l.y && j.e.ldy == l.ldy && j.e.backward == backward && j.e.act == l.act);
          }
          CHECK(p.b_kmajor == (backward == (l.w_transposed != 0)));
        }
  CHECK(tiles.size() == LIN_TILES);
  // the sizes by which the tests on the GPU mean to reach each tile
  LinPlan p;
  CHECK(run(layer(1, 768, 2304), false, &p) == MUON_OK && p.tile == LIN_TILE_32_DEEP);
  CHECK(run(layer(130, 200, 1000), false, &p) == MUON_OK && p.tile == LIN_TILE_32);
  CHECK(run(layer(1500, 72, 1304), false, &p) == MUON_OK && p.tile == LIN_TILE_64);
  CHECK(run(layer(1000, 2304, 760), false, &p) == MUON_OK && p.tile == LIN_TILE_64_DEEP);
  CHECK(run(layer(2000, 200, 1100), false, &p) == MUON_OK && p.tile == LIN_TILE_128);
  CHECK(run(layer(4097, 72, 2311), false, &p) == MUON_OK && p.tile == LIN_TILE_256x192);
  CHECK(run(layer(4160, 136, 2304), false, &p) == MUON_OK && p.tile == LIN_TILE_256x192);
  CHECK(run(layer(8200, 72, 1400), false, &p) == MUON_OK && p.tile == LIN_TILE_256);
  // and with its reduction split
  const struct {
    int64_t m, k, n;
    int tile;
  } splits[] = {{1, 4096, 72, LIN_TILE_32_DEEP}, {257, 30000, 520, LIN_TILE_64}, {64, 6400, 1600, LIN_TILE_64_DEEP}, {130, 9000, 200, LIN_TILE_32},
                {520, 20000, 1000, LIN_TILE_128}, {2048, 20000, 1032, LIN_TILE_256x192}, {1500, 20000, 1500, LIN_TILE_256}};
  for (const auto& s : splits) CHECK(run(layer(s.m, s.k, s.n), false, &p) == MUON_OK && p.finish && p.tile == s.tile);
  CHECK(run(layer(1, 768, 2304), false, &p) == MUON_OK && !p.finish);
  // a matrix that direct loads can read but for one thing: read through registers if it is
  // small, through a copy if it is large or its rows are short
  CHECK(run(layer(64, 64, 64), false, &p) == MUON_OK && p.pack.n == 0 && p.workspace == 0 && p.tile != LIN_TILE_64_ANY);
  void (*const changes[])(muon_linear_t&) = {
      [](muon_linear_t& l) { l.x = at(64, 2); },       [](muon_linear_t& l) { l.ldx += 1; },
      [](muon_linear_t& l) { l.ldx = 0; },             [](muon_linear_t& l) { l.ldx = ((int64_t)1 << 22) + 8; },
      [](muon_linear_t& l) { l.w_type = MUON_FP32; },  [](muon_linear_t& l) { l.ldw += 1; },
  };
  for (const auto& change : changes) {
    muon_linear_t l = layer(64, 64, 64);
    change(l);
    CHECK(run(l, false, &p) == MUON_OK && p.pack.n == 0 && p.workspace == 0 && p.tile == LIN_TILE_64_ANY);
    CHECK(p.b_wide == (l.w_type == MUON_FP32));
    l = layer(8192, 768, 3072);
    change(l);
    CHECK(run(l, false, &p) == MUON_OK && p.pack.n == 1 && p.workspace > 0 && p.tile != LIN_TILE_64_ANY && !p.b_wide);
  }
  for (int64_t k = 1; k <= 8; ++k) {
    CHECK(run(layer(64, k, 64), false, &p) == MUON_OK && p.pack.n == (k < 8) && p.tile != LIN_TILE_64_ANY);
    CHECK(run(layer(64, 64, k, true), true, &p) == MUON_OK && p.pack.n == (k < 8 ? 2 : 0) && p.tile != LIN_TILE_64_ANY);
  }
  muon_linear_t l;
  // no rows: nothing to do, whatever the pointers
  l = layer(0, 64, 64);
  l.x = l.y = nullptr;
  CHECK(run(l, false, &p) == MUON_OK && p.empty);
  // one row: its distance does not matter
  l = layer(1, 64, 64);
  l.ldx = 3;
  l.ldy = 0;
  CHECK(run(l, false, &p) == MUON_OK && p.pack.n == 0);
}

static void check_refusals() {
  LinPlan p;
  CHECK(said(plan_linear(nullptr, false, nullptr, 0, &p), MUON_EINVAL, "NULL"));
  struct Case {
    const char* text;
    void (*change)(muon_linear_t&);
  };
  const Case cases[] = {
      {"m = -1", [](muon_linear_t& l) { l.m = -1; }},
      {"m = 1073741825", [](muon_linear_t& l) { l.m = ((int64_t)1 << 30) + 1; }},
      {"k = 0", [](muon_linear_t& l) { l.k = 0; }},
      {"n = 0", [](muon_linear_t& l) { l.n = 0; }},
      {"n = 4194305", [](muon_linear_t& l) { l.n = (1 << 22) + 1; }},
      {"x is NULL", [](muon_linear_t& l) { l.x = nullptr; }},
      {"w is NULL", [](muon_linear_t& l) { l.w = nullptr; }},
      {"y is NULL", [](muon_linear_t& l) { l.y = nullptr; }},
      {"x is not 2-byte aligned", [](muon_linear_t& l) { l.x = at(64, 1); }},
      {"y is not 4-byte aligned", [](muon_linear_t& l) { l.y = at(192, 2), l.y_type = MUON_FP32; }},
      {"x_type = 0", [](muon_linear_t& l) { l.x_type = MUON_FP32; }},
      {"x_type = 7", [](muon_linear_t& l) { l.x_type = 7; }},
      {"w_type = 2", [](muon_linear_t& l) { l.w_type = MUON_FP16; }},
      {"y_type = 2", [](muon_linear_t& l) { l.y_type = MUON_FP16; }},
      {"bias_type = 2", [](muon_linear_t& l) { l.bias = at(300), l.bias_type = MUON_FP16; }},
      {"w_transposed = 2", [](muon_linear_t& l) { l.w_transposed = 2; }},
      {"act = 4", [](muon_linear_t& l) { l.act = 4; }},
      {"act = -1", [](muon_linear_t& l) { l.act = -1; }},
      {"dropout = 1", [](muon_linear_t& l) { l.dropout = 1.0f; }},
      {"dropout = -0.1", [](muon_linear_t& l) { l.dropout = -0.1f; }},
      {"dropout = nan", [](muon_linear_t& l) { l.dropout = std::nanf(""); }},
      {"rng is not 8-byte", [](muon_linear_t& l) { l.rng = (const int64_t*)at(300, 4), l.dropout = 0.5f; }},
      {"y: rows 63 elements apart overlap", [](muon_linear_t& l) { l.ldy = 63; }},
      {"x: rows -64 elements apart", [](muon_linear_t& l) { l.ldx = -64; }},
      {"too far", [](muon_linear_t& l) { l.ldx = (int64_t)1 << 60; }},
      {"y overlaps x", [](muon_linear_t& l) { l.y = const_cast<void*>(l.x); }},
      {"y overlaps w", [](muon_linear_t& l) { l.y = at(128, 128); }},
      {"y overlaps bias", [](muon_linear_t& l) { l.bias = at(192, 100); }},
      {"y overlaps preact", [](muon_linear_t& l) { l.preact = at(192), l.ldp = 64; }},
      {"x overlaps preact", [](muon_linear_t& l) { l.preact = at(64, 2), l.ldp = 64; }},
      {"preact overlaps residual", [](muon_linear_t& l) { l.preact = at(300), l.ldp = 64, l.residual = at(300), l.ldr = 64; }},
      {"y overlaps residual", [](muon_linear_t& l) { l.residual = at(192, 2), l.ldr = 64; }},
      {"y overlaps rng", [](muon_linear_t& l) { l.rng = (const int64_t*)at(192, 8), l.dropout = 0.5f; }},
      {"workspace overlaps x", [](muon_linear_t& l) { l.k = 7, l.x = at(512, 2); }},
      {"workspace overlaps w", [](muon_linear_t& l) { l.k = 7, l.w = at(512), l.w_type = MUON_FP32; }},
  };
  for (const Case& c : cases) {
    muon_linear_t l = layer(64, 64, 64);
    c.change(l);
    CHECK(said(run(l), MUON_EINVAL, c.text));
  }
  // the gradient of the input
  muon_linear_t l = layer(64, 64, 64, true);
  l.bias = at(300);
  CHECK(said(run(l, true), MUON_EINVAL, "takes no bias"));
  l = layer(64, 64, 64, true);
  l.act = MUON_ACT_GELU;
  CHECK(said(run(l, true), MUON_EINVAL, "come together"));
  l.act = MUON_ACT_NONE;
  l.preact = at(300);
  l.ldp = 64;
  CHECK(said(run(l, true), MUON_EINVAL, "come together"));
  l.act = MUON_ACT_RELU;
  CHECK(run(l, true) == MUON_OK);
  l.preact = l.y;  // in place
  CHECK(run(l, true) == MUON_OK);
  l.residual = l.y;
  l.ldr = 64;
  CHECK(run(l, true) == MUON_OK);
  l.preact = at(192, 64);
  CHECK(said(run(l, true), MUON_EINVAL, "y overlaps preact"));
  // the residual in place, another distance or type not
  l = layer(64, 64, 64);
  l.residual = l.y;
  l.ldr = 64;
  CHECK(run(l) == MUON_OK);
  l.ldr = 65;
  CHECK(said(run(l), MUON_EINVAL, "y overlaps residual"));
  // column ranges of one buffer
  l = layer(64, 64, 64);
  l.ldx = l.ldy = 200;
  l.y = at(64, 64 * 2);
  CHECK(run(l) == MUON_OK);
  l.y = at(64, 136 * 2);
  CHECK(run(l) == MUON_OK);
  l.y = at(64, 137 * 2);
  CHECK(said(run(l), MUON_EINVAL, "y overlaps x"));
  l.y = at(64, 63 * 2);
  CHECK(said(run(l), MUON_EINVAL, "y overlaps x"));
  l.x = at(64, 137 * 2);
  l.y = at(64);
  CHECK(said(run(l), MUON_EINVAL, "y overlaps x"));
  l.x = at(64, 136 * 2);
  CHECK(run(l) == MUON_OK);
  // the workspace
  l = layer(64, 7, 64);
  size_t bytes = 0;
  CHECK(linear_workspace(&l, false, &bytes) == MUON_OK && bytes >= 64 * 8 * 2);
  CHECK(said(plan_linear(&l, false, nullptr, bytes, &p), MUON_EINVAL, "workspace is NULL"));
  CHECK(said(plan_linear(&l, false, at(512, 8), bytes, &p), MUON_EINVAL, "16-byte"));
  CHECK(said(plan_linear(&l, false, at(512), bytes - 1, &p), MUON_ENOMEM, "needs"));
  CHECK(plan_linear(&l, false, at(512), bytes, &p) == MUON_OK);
  l.n = 0;
  CHECK(linear_workspace(&l, false, &bytes) == MUON_EINVAL && bytes == 0);
  // the most rows
  l = layer((int64_t)1 << 30, 8, 8);
  CHECK(said(run(l), MUON_EINVAL, "too large") || run(l) == MUON_OK);
}

static muon_linear_dw_t grad(int64_t m, int64_t k, int64_t n, int t = 0) {
  muon_linear_dw_t l = {};
  l.m = m;
  l.k = k;
  l.n = n;
  l.x = at(64);
  l.dz = at(128);
  l.dw = (float*)at(192);
  l.dbias = (float*)at(256);
  l.ldx = k;
  l.lddz = n;
  l.lddw = t ? k : n;
  l.type = MUON_FP16;
  l.dw_transposed = t;
  return l;
}

static int run(const muon_linear_dw_t& l, LinPlan* out = nullptr) {
  LinPlan p;
  size_t bytes = 0;
  linear_dw_workspace(&l, &bytes);
  return plan_linear_dw(&l, at(512), bytes, out ? out : &p);
}

static void check_grads() {
  std::set<int> tiles;
  bool split = false;
  for (int64_t m : {0, 1, 64, 515, 4100, 16384, 300000})
    for (int64_t k : {1, 8, 333, 768, 4096})
      for (int64_t n : {1, 40, 1001, 2304})
        for (int v = 0; v < 8; ++v) {
          muon_linear_dw_t l = grad(m, k, n, v & 1);
          l.accumulate = (v >> 1) & 1;
          if (v & 4) l.dbias = nullptr;
          LinPlan p;
          CHECK(run(l, &p) == MUON_OK);
          CHECK(p.empty == (m == 0 && l.accumulate));
          if (p.empty) continue;
          check_gemm(p, v & 1 ? n : k, v & 1 ? k : n, m);
          tiles.insert(p.tile);
          split = split || p.finish;
          CHECK(p.finish == (p.gemm.splits > 1));
          CHECK(p.gemm.sum_side == (v & 4 ? 0 : v & 1 ? 2 : 1));
          if (p.finish) {
            const LinTileSize t = kLinTile[p.tile];
            const LinFinishArgs& f = p.fin;
            CHECK(f.part_ld == (int64_t)p.gemm.tiles_n * t.bn && f.part_stride == f.part_ld * p.gemm.tiles_m * t.bm);
            const char* end = (const char*)at(512) + p.workspace;
            CHECK((const char*)(f.part + f.part_stride * f.splits) <= end && f.part_ld >= (f.n + 7) / 8 * 8);
            CHECK((int64_t)f.sum_first_block * FINISH_THREADS >= (int64_t)f.m * ((f.n + 7) / 8));
            if (p.gemm.sum_side) {
              CHECK((const char*)(f.sum_part + f.sum_stride * f.sum_rows) <= end && f.sum_part >= f.part + f.part_stride * f.splits);
              CHECK(f.sum_stride >= f.n_sums && f.sum_rows == f.splits * (p.gemm.sum_side == 1 ? p.gemm.tiles_m : p.gemm.tiles_n));
            }
          }
        }
  CHECK(split && tiles.size() == 5 && !tiles.count(LIN_TILE_32) && !tiles.count(LIN_TILE_64_DEEP));
  LinPlan p;
  CHECK(run(grad(72, 4097, 2311), &p) == MUON_OK && p.tile == LIN_TILE_256x192);
  CHECK(run(grad(72, 8200, 1400), &p) == MUON_OK && p.tile == LIN_TILE_256);
  CHECK(run(grad(200, 2000, 1100), &p) == MUON_OK && p.tile == LIN_TILE_128);
  CHECK(run(grad(4100, 72, 200), &p) == MUON_OK && p.finish);
  CHECK(run(grad(30000, 520, 264), &p) == MUON_OK && p.finish);

  struct Case {
    const char* text;
    void (*change)(muon_linear_dw_t&);
  };
  const Case cases[] = {
      {"m = -1", [](muon_linear_dw_t& l) { l.m = -1; }},
      {"k = 0", [](muon_linear_dw_t& l) { l.k = 0; }},
      {"n = 0", [](muon_linear_dw_t& l) { l.n = 0; }},
      {"type = 0", [](muon_linear_dw_t& l) { l.type = MUON_FP32; }},
      {"dw_transposed = 3", [](muon_linear_dw_t& l) { l.dw_transposed = 3; }},
      {"accumulate = 2", [](muon_linear_dw_t& l) { l.accumulate = 2; }},
      {"x is NULL", [](muon_linear_dw_t& l) { l.x = nullptr; }},
      {"dz is NULL", [](muon_linear_dw_t& l) { l.dz = nullptr; }},
      {"dw is NULL", [](muon_linear_dw_t& l) { l.dw = nullptr; }},
      {"dw is not 4-byte", [](muon_linear_dw_t& l) { l.dw = (float*)at(192, 2); }},
      {"dbias is not 4-byte", [](muon_linear_dw_t& l) { l.dbias = (float*)at(256, 2); }},
      {"dw: rows 63 elements apart overlap", [](muon_linear_dw_t& l) { l.lddw = 63; }},
      {"dw overlaps dbias", [](muon_linear_dw_t& l) { l.dbias = (float*)at(192, 128); }},
      {"dw overlaps x", [](muon_linear_dw_t& l) { l.x = at(192); }},
      {"dbias overlaps dz", [](muon_linear_dw_t& l) { l.dz = at(256); }},
  };
  for (const Case& c : cases) {
    muon_linear_dw_t l = grad(64, 64, 64);
    c.change(l);
    CHECK(said(run(l), MUON_EINVAL, c.text));
  }
  CHECK(said(plan_linear_dw(nullptr, nullptr, 0, &p), MUON_EINVAL, "NULL"));
  // x and dz may be one matrix
  muon_linear_dw_t l = grad(64, 64, 64);
  l.dz = l.x;
  CHECK(run(l) == MUON_OK);
  l = grad(20000, 64, 64);
  CHECK(said(plan_linear_dw(&l, at(512), 16, &p), MUON_ENOMEM, "needs"));
}

static void check_dropout() {
  DropArgs a;
  int64_t blocks = -1;
  muon_dropout_t d = {};
  d.m = 37;
  d.n = 131;
  d.x = at(64);
  d.y = at(128);
  d.ldx = d.ldy = d.ldp = d.ldr = 131;
  d.x_type = MUON_FP32;
  d.y_type = MUON_BF16;
  d.dropout = 0.1f;
  CHECK(plan_dropout(&d, &a, &blocks) == MUON_OK && blocks == 3 && a.e.border == 6554);  // 37 x 17 eights
  struct {
    float p;
    uint32_t border;
  } const borders[] = {{0.0f, 0}, {7.6e-6f, 0}, {7.7e-6f, 1}, {0.5f, 32768}, {0.99999f, 65535}, {1 - 0x1p-24f, 65535}};
  for (const auto& b : borders) {
    d.dropout = b.p;
    CHECK(plan_dropout(&d, &a, &blocks) == MUON_OK && a.e.border == b.border);
    CHECK(a.e.keep_scale == (float)(65536.0 / (65536.0 - b.border)));
  }
  auto refused = [&](const muon_dropout_t& v, const char* text) { return said(plan_dropout(&v, &a, &blocks), MUON_EINVAL, text); };
  CHECK(said(plan_dropout(nullptr, &a, &blocks), MUON_EINVAL, "NULL"));
  muon_dropout_t v = d;
  v.dropout = 1.0f;
  CHECK(refused(v, "dropout = 1"));
  v = d, v.m = -1;
  CHECK(refused(v, "m = -1"));
  v = d, v.n = ((int64_t)1 << 34) + 1;
  CHECK(refused(v, "n = "));
  v = d, v.x = nullptr;
  CHECK(refused(v, "x is NULL"));
  v = d, v.x_type = 3;
  CHECK(refused(v, "x_type = 3"));
  v = d, v.y_type = -1;
  CHECK(refused(v, "y_type = -1"));
  v = d, v.act = MUON_ACT_GELU;
  CHECK(refused(v, "come together"));
  v = d, v.preact = at(300);
  CHECK(refused(v, "come together"));
  v = d, v.ldy = 130;
  CHECK(refused(v, "overlap"));
  v = d, v.y = at(64);
  CHECK(refused(v, "y overlaps x"));  // another type
  v.y_type = MUON_FP32;
  CHECK(plan_dropout(&v, &a, &blocks) == MUON_OK);
  v = d, v.residual = at(128, 2);
  CHECK(refused(v, "y overlaps residual"));
  v.residual = at(128);
  CHECK(plan_dropout(&v, &a, &blocks) == MUON_OK);
  v = d, v.m = (int64_t)1 << 30, v.n = (int64_t)1 << 12;
  v.ldx = v.ldy = v.n;
  v.y = at((uint64_t)1 << 20);
  CHECK(refused(v, "too many"));
  for (int64_t m : {0, 5})
    for (int64_t n : {0, 5})
      if (m * n == 0) {
        v = d, v.m = m, v.n = n, v.x = nullptr;
        CHECK(plan_dropout(&v, &a, &blocks) == MUON_OK && blocks == 0);
      }
}

int main() {
  check_layers();
  check_refusals();
  check_grads();
  check_dropout();
  if (g_failures) return 1;
  std::puts("ok");
  return 0;
}
