// Host check of what the layer products take at the limits of a launch
// (csrc/linear_host.cpp, linear_types.h): tiles that a grid cannot hold are passed
// over for others, and copies of more blocks than a launch has go out in several.  Built and run by tests/test_linear_limits.py, under
// sanitizers.  Prints "ok" and exits 0 when every check holds.
#include <cstdio>
#include <limits>
#include <string>
#include <vector>

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

// Addresses are only compared, never followed.
static void* at(uint64_t tib) { return (void*)(uintptr_t)(tib << 40); }

static muon_linear_t layer(int64_t m, int64_t k, int64_t n) {
  muon_linear_t l = {};
  l.m = m;
  l.k = k;
  l.n = n;
  l.x = at(1);
  l.w = at(2);
  l.y = at(3);
  l.ldx = k;
  l.ldw = l.ldy = n;
  l.x_type = l.w_type = l.y_type = MUON_BF16;
  return l;
}

static muon_linear_dw_t grad(int64_t m, int64_t k, int64_t n) {
  muon_linear_dw_t l = {};
  l.m = m;
  l.k = k;
  l.n = n;
  l.x = at(1);
  l.dz = at(2);
  l.dw = (float*)at(3);
  l.ldx = k;
  l.lddz = l.lddw = n;
  l.type = MUON_FP16;
  return l;
}

static int run(const muon_linear_t& l, LinPlan* out) {
  size_t bytes = 0;
  linear_workspace(&l, false, &bytes);
  const int rc = plan_linear(&l, false, at(16), bytes, out);
  if (rc) std::fprintf(stderr, "  %lld x %lld x %lld: %s\n", (long long)l.m, (long long)l.k, (long long)l.n, last_error_text());
  return rc;
}

static int run(const muon_linear_dw_t& l, LinPlan* out) {
  size_t bytes = 0;
  linear_dw_workspace(&l, &bytes);
  const int rc = plan_linear_dw(&l, at(16), bytes, out);
  if (rc) std::fprintf(stderr, "  dw %lld x %lld x %lld: %s\n", (long long)l.m, (long long)l.k, (long long)l.n, last_error_text());
  return rc;
}

static int64_t copied_blocks(const LinPlan& p) {
  int64_t blocks = 0;
  for (int i = 0; i < p.pack.n; ++i) blocks += pack_blocks(p.pack.job[i]);
  return blocks;
}

// Copies below, at and above the blocks of one launch.
static void check_copies() {
  LinPlan p;
  // 256 rows of 128 are 16 blocks: the last whole launch ends at 2^28 - 16 rows
  for (int64_t m : {((int64_t)1 << 28) - 16, (int64_t)1 << 28, ((int64_t)1 << 28) + 1}) {
    CHECK(run(layer(m, 127, 192), &p) == MUON_OK);
    CHECK(run(grad(m, 127, 5), &p) == MUON_OK && p.pack.n == 2 && copied_blocks(p) > MAX_LAUNCH_ITEMS);
    CHECK(p.workspace >= (size_t)m * (128 + 8) * 2);
  }
  for (int64_t blocks : {(int64_t)0, (int64_t)1, MAX_LAUNCH_ITEMS - 1, MAX_LAUNCH_ITEMS, MAX_LAUNCH_ITEMS + 1, 5 * MAX_LAUNCH_ITEMS,
                         5 * MAX_LAUNCH_ITEMS + 7}) {
    int64_t next = 0;
    std::vector<int> launches;
    const int rc = for_launches(blocks, [&](int64_t first, int n) {
      CHECK(first == next && n > 0 && n <= MAX_LAUNCH_ITEMS);
      next = first + n;
      launches.push_back(n);
      return 0;
    });
    CHECK(rc == 0 && next == blocks && (int64_t)launches.size() == (blocks + MAX_LAUNCH_ITEMS - 1) / MAX_LAUNCH_ITEMS);
  }
  int calls = 0;
  CHECK(for_launches(3 * MAX_LAUNCH_ITEMS, [&](int64_t, int) { return ++calls == 2 ? 7 : 0; }) == 7 && calls == 2);
}

// A grid holds fewer than 2^32 threads.
static void check_grid(const LinPlan& p, int64_t m, int64_t n) {
  const LinTileSize t = kLinTile[p.tile];
  CHECK((int64_t)p.gemm.tiles_m * p.gemm.tiles_n * p.gemm.splits * t.threads < (int64_t)1 << 32);
  CHECK((int64_t)p.gemm.tiles_m * t.bm >= m && (int64_t)p.gemm.tiles_n * t.bn >= n);
}

static void check_grids() {
  LinPlan p;
  const int64_t most = (int64_t)1 << 30;
  // the most rows, short enough to be read where they lie
  CHECK(run(layer(most, 8, 8), &p) == MUON_OK && p.pack.n == 0 && p.workspace == 0 && p.tile == LIN_TILE_256x192);
  check_grid(p, most, 8);
  // the last row count whose 64 x 64 tiles of 512 threads a grid holds, and the first beyond it
  const int64_t last = (((int64_t)1 << 23) - 1) * 64;
  CHECK(run(layer(last, 61, 8), &p) == MUON_OK && p.tile == LIN_TILE_64_ANY && p.pack.n == 0);
  check_grid(p, last, 8);
  CHECK(run(layer(last + 1, 61, 8), &p) == MUON_OK && p.tile != LIN_TILE_64_ANY && p.pack.n == 1);
  check_grid(p, last + 1, 8);
  for (int64_t m : {((int64_t)1 << 28) + 1, ((int64_t)1 << 29) - 1, (int64_t)1 << 29, most - 1, most})
    for (int64_t k : {1, 8, 25, 57, 61, 64, 127})
      for (int64_t n : {1, 8, 61, 64, 192, 256}) {
        CHECK(run(layer(m, k, n), &p) == MUON_OK);
        check_grid(p, m, n);
      }
  for (int64_t k : {(int64_t)1 << 20, (int64_t)1 << 22})
    for (int64_t n : {100, 1000, 100000}) {
      CHECK(run(grad(100, k, n), &p) == MUON_OK);
      check_grid(p, k, n);
    }
  // 2^23 tiles of 256 x 256, more than any device's memory: refused
  CHECK(run(layer(most - 255, 64, 256), &p) == MUON_OK);
  CHECK(run(layer(most, 64, 257), &p) == MUON_EINVAL && std::string(last_error_text()).find("too large") != std::string::npos);
  CHECK(run(grad(64, (int64_t)1 << 22, (int64_t)1 << 22), &p) == MUON_EINVAL);
  size_t bytes = 1;
  const muon_linear_t l = layer(most, 64, 257);
  CHECK(linear_workspace(&l, false, &bytes) == MUON_EINVAL && bytes == 0);
}

// The sizes by which tests/test_gpu_linear_long.py means to reach each tile, split and not,
// over more slices than any ring holds.
static void check_long() {
  LinPlan p;
  const struct {
    int64_t m, k, n;
    int tile;
    bool split;
  } layers[] = {{8200, 1608, 1400, LIN_TILE_256, false},     {1504, 20000, 1504, LIN_TILE_256, true},
                {4160, 1608, 2304, LIN_TILE_256x192, false}, {2048, 20000, 1032, LIN_TILE_256x192, true},
                {2000, 1608, 1104, LIN_TILE_128, false},     {520, 20000, 1000, LIN_TILE_128, true},
                {1500, 1608, 1304, LIN_TILE_64, false},      {257, 30000, 520, LIN_TILE_64, true},
                {1000, 2312, 760, LIN_TILE_64_DEEP, false},  {64, 6408, 1600, LIN_TILE_64_DEEP, true},
                {130, 1608, 1000, LIN_TILE_32, false},       {130, 9000, 200, LIN_TILE_32, true},
                {20, 1608, 16000, LIN_TILE_32_DEEP, false},  {1, 4104, 2304, LIN_TILE_32_DEEP, true},
                {700, 1001, 1003, LIN_TILE_64_ANY, false},   {257, 30001, 513, LIN_TILE_64_ANY, true}},
    grads[] = {{3000, 8200, 1400, LIN_TILE_256, false},     {20000, 1400, 2040, LIN_TILE_256, true},
               {3000, 4160, 2304, LIN_TILE_256x192, false}, {16384, 768, 2304, LIN_TILE_256x192, true},
               {4000, 2504, 1304, LIN_TILE_128, false},     {3000, 2000, 1104, LIN_TILE_128, true},
               {4000, 1504, 1304, LIN_TILE_64, false},      {30000, 520, 264, LIN_TILE_64, true},
               {2004, 333, 2001, LIN_TILE_64_ANY, false},   {3001, 131, 300, LIN_TILE_64_ANY, true}};
  for (const auto& s : layers) {
    CHECK(run(layer(s.m, s.k, s.n), &p) == MUON_OK && p.tile == s.tile && p.finish == s.split);
    CHECK(p.pack.n == 0 && p.gemm.slices >= 8);
  }
  for (const auto& s : grads)
    for (int t : {0, 1}) {  // stored the other way the roles of x and dz change places
      muon_linear_dw_t l = grad(s.m, t ? s.n : s.k, t ? s.k : s.n);
      l.dw_transposed = t;
      l.lddw = t ? l.k : l.n;
      l.dbias = (float*)at(4);
      CHECK(run(l, &p) == MUON_OK && p.tile == s.tile && p.finish == s.split);
      CHECK(p.pack.n == 0 && p.gemm.slices >= 8 && p.gemm.sum_side == 1 + t);
    }
  CHECK(run(layer(4097, 1609, 2311), &p) == MUON_OK && p.pack.n == 2 && p.tile == LIN_TILE_256x192);
  CHECK(run(grad(20001, 1001, 771), &p) == MUON_OK && p.pack.n == 2 && p.finish);
}

// The distance between rows of a matrix of one row means nothing, whatever it is.
static void check_one_row() {
  const int64_t any[] = {0, 3, -1, std::numeric_limits<int64_t>::max(), std::numeric_limits<int64_t>::min()};
  for (int64_t k : {1, 8, 61, 768})
    for (int64_t n : {1, 61, 768, 6400})
      for (int type : {MUON_BF16, MUON_FP32}) {
        muon_linear_t l = layer(1, k, n);
        l.w_type = type;
        l.preact = at(4);
        l.residual = at(5);
        l.ldp = l.ldr = n;
        LinPlan want, p;
        CHECK(run(l, &want) == MUON_OK);
        for (int64_t ld : any) {
          l.ldx = l.ldy = l.ldp = l.ldr = ld;
          if (k == 1) l.ldw = ld;
          CHECK(run(l, &p) == MUON_OK && p.tile == want.tile && p.gemm.splits == want.gemm.splits);
          CHECK(p.gemm.a.ld == want.gemm.a.ld && p.gemm.b.ld == want.gemm.b.ld && p.workspace == want.workspace);
        }
        muon_linear_dw_t g = grad(1, k, n);
        CHECK(run(g, &want) == MUON_OK);
        for (int64_t ld : any) {
          g.ldx = g.lddz = ld;
          if (k == 1) g.lddw = ld;
          CHECK(run(g, &p) == MUON_OK && p.tile == want.tile && p.gemm.a.ld == want.gemm.a.ld && p.gemm.b.ld == want.gemm.b.ld);
        }
      }
}

// The size of a workspace is asked for before there are buffers: pointers may be anything,
// the distances of what is read not.
static void check_sizes() {
  for (int64_t ld : {std::numeric_limits<int64_t>::max(), std::numeric_limits<int64_t>::min(), (int64_t)-1, (int64_t)1 << 60}) {
    size_t bytes = 1;
    muon_linear_t l = layer(64, 61, 64);
    l.x = l.w = l.y = nullptr;
    l.ldx = ld;
    CHECK(linear_workspace(&l, false, &bytes) == MUON_EINVAL && bytes == 0);
    l.ldx = 61;
    l.ldw = ld;
    CHECK(linear_workspace(&l, true, &bytes) == MUON_EINVAL && bytes == 0);
    l.ldw = 64;
    l.ldy = ld;  // the size does not go by it
    CHECK(linear_workspace(&l, false, &bytes) == MUON_OK);
    muon_linear_dw_t g = grad(64, 61, 64);
    g.x = g.dz = nullptr;
    g.dw = nullptr;
    g.lddz = ld;
    CHECK(linear_dw_workspace(&g, &bytes) == MUON_EINVAL && bytes == 0);
    g.lddz = 64;
    CHECK(linear_dw_workspace(&g, &bytes) == MUON_OK);
  }
}

// Up to 32 rows: the deep ring while every tile has a unit to itself, two tiles to a unit beyond.
static void check_few_rows() {
  LinPlan p;
  for (int64_t m : {1, 8, 32}) {
    CHECK(run(layer(m, 768, 16384), &p) == MUON_OK && p.tile == LIN_TILE_32_DEEP && p.gemm.tiles_n == 256);
    for (int64_t n : {16392, 20000, 32768, 50264, 100000})
      CHECK(run(layer(m, 768, n), &p) == MUON_OK && p.tile == LIN_TILE_32 && p.gemm.tiles_n > 256);
    muon_linear_t l = layer(m, 768, 50257);  // a vocabulary of the framework's, stored out x in
    l.w_transposed = 1;
    l.ldw = 768;
    CHECK(run(l, &p) == MUON_OK && p.tile == LIN_TILE_32 && p.pack.n == 0);
  }
}

int main() {
  check_few_rows();
  check_sizes();
  check_one_row();
  check_long();
  check_grids();
  check_copies();
  if (g_failures) return 1;
  std::puts("ok");
  return 0;
}
