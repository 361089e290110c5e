// Validation and launch arguments of the hidden layers' products and of
// dropout.  No GPU calls.
#include "linear_host.h"

#include <algorithm>
#include <cmath>

#include "plan_host.h"

namespace muon {

static_assert(LIN_ACT_NONE == MUON_ACT_NONE && LIN_ACT_GELU == MUON_ACT_GELU && LIN_ACT_RELU == MUON_ACT_RELU &&
                  LIN_ACT_RELU2 == MUON_ACT_RELU2, "activation codes");

namespace {

constexpr int64_t MAX_WIDTH = MUON_LINEAR_MAX_WIDTH;
constexpr int64_t MAX_ROWS = MUON_LINEAR_MAX_ROWS;
constexpr int64_t MAX_BYTES = (int64_t)1 << 46;  // of one matrix, gaps between its rows included

// A matrix of a call: rows of `cols` elements, ld elements apart.
struct Matrix {
  const char* what;
  const void* p;
  int64_t rows, cols, ld;
  int type;
  bool written;

  uintptr_t lo() const { return (uintptr_t)p; }
  uint64_t size() const { return grad_type_bytes(type); }
  int64_t pitch() const { return rows == 1 ? cols : ld; }  // that of one row is not given
  uintptr_t hi() const { return lo() + (uint64_t)((rows - 1) * ld + cols) * size(); }
  bool is(const Matrix& o) const { return p == o.p && type == o.type && (ld == o.ld || rows == 1); }
};

int check_dim(int64_t v, int64_t least, int64_t most, const char* what) {
  if (v < least || v > most)
    return fail(MUON_EINVAL, "%s = %lld outside [%lld, %lld]", what, (long long)v, (long long)least, (long long)most);
  return MUON_OK;
}

int check_matrix(const Matrix& m, bool sizes_only = false) {
  if (m.type < MUON_FP32 || m.type > MUON_FP16)
    return fail(MUON_EINVAL, "%s: type %d is no element type (MUON_FP32, MUON_BF16, MUON_FP16)", m.what, m.type);
  if (!m.p && !sizes_only) return fail(MUON_EINVAL, "%s is NULL", m.what);
  if (m.lo() % m.size() && !sizes_only) return fail(MUON_EINVAL, "%s is not %d-byte aligned", m.what, (int)m.size());
  if (m.rows > 1 && (m.written ? m.ld < m.cols : m.ld < 0))
    return fail(MUON_EINVAL, "%s: rows %lld elements apart%s", m.what, (long long)m.ld,
                m.written ? " overlap" : "");
  if (m.rows > 1 && m.ld > MAX_BYTES / 4 / m.rows)
    return fail(MUON_EINVAL, "%s: rows %lld elements apart are too far", m.what, (long long)m.ld);
  return MUON_OK;
}

// Two matrices that share an element.  Column ranges of one buffer do not.
bool overlap(const Matrix& a, const Matrix& b) {
  if (a.lo() >= b.hi() || b.lo() >= a.hi()) return false;
  const uint64_t wa = (uint64_t)a.cols * a.size(), wb = (uint64_t)b.cols * b.size();
  const uint64_t la = (uint64_t)a.ld * a.size(), lb = (uint64_t)b.ld * b.size();
  const uint64_t pitch = a.rows > 1 ? la : lb;
  if ((a.rows > 1 && b.rows > 1 && la != lb) || pitch < wa || pitch < wb) return true;
  const uint64_t apart = b.lo() >= a.lo() ? (b.lo() - a.lo()) % pitch : (pitch - (a.lo() - b.lo()) % pitch) % pitch;
  return apart < wa || apart + wb > pitch;
}

// Written matrices against all others; `may_be[i]`: matrix i may be matrix 0 itself.
int check_overlaps(const Matrix* m, const bool* may_be_first, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (!m[i].written && !m[j].written) continue;
      if (i == 0 && may_be_first[j] && m[0].is(m[j])) continue;
      if (overlap(m[i], m[j])) return fail(MUON_EINVAL, "%s overlaps %s", m[i].what, m[j].what);
    }
  return MUON_OK;
}

int check_epilogue(int act, float dropout, const int64_t* rng) {
  if (act < MUON_ACT_NONE || act > MUON_ACT_RELU2) return fail(MUON_EINVAL, "act = %d is no activation", act);
  if (!(dropout >= 0.0f && dropout < 1.0f)) return fail(MUON_EINVAL, "dropout = %g outside [0, 1)", (double)dropout);
  if ((uintptr_t)rng % 8) return fail(MUON_EINVAL, "rng is not 8-byte aligned");
  return MUON_OK;
}

void fill_dropout(LinEpilogue* e, float p, uint64_t seed, uint32_t step, uint32_t site, const int64_t* rng) {
  e->border = std::min((uint32_t)std::floor(65536.0 * (double)p + 0.5), 65535u);
  e->keep_scale = (float)(65536.0 / (65536.0 - e->border));
  e->seed = seed;
  e->step = step;
  e->site = site;
  e->rng = rng;
}

// Whether the kernels can read a matrix in place.
bool readable(const Matrix& m, int type) {
  return m.type == type && m.lo() % 16 == 0 && m.cols % 8 == 0 &&
         (m.rows == 1 || (m.ld % 8 == 0 && m.ld >= m.cols && m.ld <= MAX_WIDTH));
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Takes `bytes` from the workspace.
char* take(LinPlan* p, void* workspace, size_t bytes) {
  const uintptr_t at = (uintptr_t)workspace + p->workspace;
  p->workspace += round_up(bytes, 256);
  return (char*)at;
}

// The operand that the kernels read for m, through a copy where they must.
LinOperand operand_of(const Matrix& m, int type, LinPlan* plan, void* workspace) {
  if (plan->tile == LIN_TILE_64_ANY) return {m.p, m.pitch() * (int64_t)m.size(), 0};
  if (readable(m, type)) return {m.p, m.pitch() * 2, ((m.rows - 1) * m.pitch() + m.cols) * 2};
  const int64_t ld = (m.cols + 7) / 8 * 8;
  char* dst = take(plan, workspace, (size_t)(m.rows * ld * 2));
  plan->pack.job[plan->pack.n++] = {m.p, dst, m.pitch(), ld, m.rows, m.cols, m.type, type};
  return {dst, ld * 2, m.rows * ld * 2};
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Microseconds of a round of tiles over the 256 compute units, as measured (bf16, one MI355X):
// a start and an end and so much for each 64 of K; one tile to a unit, or the two
// that small tiles leave room for.  Over a K of 768 a round of 256 x 256 tiles
// takes 26.6, of 256 x 192 21.8, of 128 x 128 13.2 and 19, of 64 x 64 6.2 and 8.8, of 32 x 64 5.3 and
// 6.9; over 3072 77, 64, 35 and 49, 14 and 22, 12 and 16.  Two k-major operands (a weight
// gradient's) take 1.17 of that a slice, except in 256 x 192 tiles, and rows that do not start at
// multiples of 16 bytes, loaded through registers, 1.45.
struct TileCost {
  double one, one_slice, two, two_slice;  // two = 0: no second tile fits
};
constexpr TileCost kTileCost[LIN_TILES] = {
    {9.7, 1.41, 0, 0}, {7.6, 1.18, 0, 0}, {6.0, 0.6, 9.0, 0.83}, {3.6, 0.23, 4.5, 0.36}, {3.7, 0.205, 0, 0}, {3.1, 0.185, 4.0, 0.24}, {3.1, 0.185, 0, 0},
    {4.0, 0.27, 5.0, 0.46}};
constexpr double GRAD_SLICE = 1.17, UNALIGNED_SLICE = 1.45;

double tiles_us(int tile, int64_t tiles, double slices) {
  const TileCost& c = kTileCost[tile];
  const double one = c.one + c.one_slice * slices, two = c.two + c.two_slice * slices;
  if (c.two == 0) return (double)((tiles + 255) / 256) * one;
  const int64_t rest = tiles % 512;
  return (double)(tiles / 512) * two + (rest > 256 ? two : rest > 0 ? one : 0);
}

// A split leaves its sums in memory and a last pass adds them up: 3 us for the
// launch, and the sums written and read at 5 TB/s.  For a layer of few rows with a bias (us in a graph,
// three sets of operands in turn, with and without splits): 1 x 768 over 3072 7.0 and 12.6,
// 64 x 1600 over 6400 13.2 and 22.1, 2048 x 1600 over 6400 62 and 71 (one set: 57 and 70);
// 1 x 2304 over 768 is not split, 5.4.
double splits_us(int64_t m, int64_t n, int64_t splits) { return splits == 1 ? 0 : 3.0 + (double)(m * n * splits) * 8 / 5e6; }

// The copies that operands need in all tiles but 64_ANY: 3 us for the launch, their
// bytes at 4 TB/s.
struct Copies {
  double us = 0;
  bool avoidable = false;  // there are some, and 64_ANY can do without
  bool unaligned = false;
  Copies(const Matrix& a, const Matrix& b, int type) {
    for (const Matrix* m : {&a, &b}) {
      if (m->rows == 0) return;
      if (!readable(*m, type)) us += (double)(m->rows * m->cols) * (double)(m->size() + 2) / 4e6;
      unaligned = unaligned || m->lo() % 16 != 0 || m->pitch() * (int64_t)m->size() % 16 != 0;
    }
    if (us == 0) return;
    us += 3.0;
    avoidable = a.cols >= 8 && b.cols >= 8;
  }
};

// Tiles, slices and splits of a product: what the measured times make the
// fastest.  The times leave the epilogue out, whose loads and stores cost all tiles about the same.
// Examples (us, forward with a bias, bf16, in a graph, three sets of operands in turn; chosen and next):
// 16384 x 3072 over 768 85 in 256 x 256 tiles, 92 in 256 x 192 (with GELU 94 and 102, with z
// kept too 103 and 112); 16384 x 768 over 3072 78 in 256 x 192 (256 tiles, one to a unit), 87 in
// 256 x 256 (with dropout and residual 83 and 91); 4096 x 768 over 768 12.9 in 128 x 128, 19.6 in 256 x 192;
// 1024 x 768 over 2304 11.5 in 64 x 64 with the deep ring, 14.7 with the other, 20
// in 128 x 128; 512 x 768 over 3072 12.5 in 32 x 64, 15.6 in 64 x 64.
//
// 64_ANY stands against the copies and any other tile.  Of an fp32 weight (the same form): 1 x 2304
// over 768 6.9 us in it and 9.3 with the copy, 4096 x 768 over 768 18.5 and 16.3, 16384 x 3072
// over 768 231 and 87.  1999 x 771 over 1001, fp16: 18.8 and 20.7, of an fp32 weight 20.2 and
// 20.0, where the copy's launch and workspace cost a call 4 us on the host besides.
int lay_out(LinPlan* p, int64_t m, int64_t n, int64_t k, bool grad, const Copies& copies) {
  LinGemmArgs& g = p->gemm;
  g.m = (int32_t)m;
  g.n = (int32_t)n;
  g.k = (int32_t)k;
  double best = 0;
  for (int tile = 0; tile < LIN_TILES; ++tile) {
    // few rows of a weight, or few weights over few rows, are no case worth a kernel
    if (grad && (tile == LIN_TILE_32 || tile == LIN_TILE_64_DEEP || tile == LIN_TILE_32_DEEP)) continue;
    if (tile == LIN_TILE_64_ANY && !copies.avoidable) continue;
    const bool any = tile == LIN_TILE_64_ANY;
    const double slower = (grad && tile != LIN_TILE_256x192 ? GRAD_SLICE : 1.0) * (any && copies.unaligned ? UNALIGNED_SLICE : 1.0);
    const LinTileSize t = kLinTile[tile];
    const int64_t tm = (m + t.bm - 1) / t.bm, tn = (n + t.bn - 1) / t.bn, tiles = tm * tn;
    // Up to 32 rows take 32 x 64 tiles with either ring, which cost the same while every tile has a unit to
    // itself; the deep one is taken there.  One row of 2304 over 768, 1600 and 3072, the weight's rows
    // along K: read from HBM 5.8, 8.8 and 13.1 us with the deep ring, 5.8, 8.8 and 13.3 with the other;
    // from the caches 5.5, 8.4 and 12.8, and 5.3, 8.0 and 12.3.  Beyond, the other fits twice into a unit:
    // one row of 50257 over 768, from HBM (from the caches), 19.2 us (16.1) with it, 24.3 (21.9) with the
    // deep ring, 21.2 (16.7) in 64 x 64; of 20000 10.6 (9.2), 13.3 (12.2) and 11.4 (9.0).  Over the
    // measured shapes it takes 4 % less than 64 x 64 in sum from HBM and 1 % less from the caches; it loses most for
    // 32768 over 3072 with the weight's rows along the columns, 51.1 to 47.7 (43.8 to 38.7).
    if (tile == LIN_TILE_32 && m <= 32 && tiles <= 256) continue;
    const int slices = ceil_div(k, t.bk);
    for (int fill = 0; fill <= 2; ++fill) {  // no splits, or as many as make one or two rounds
      const int64_t want = fill == 0 ? 1 : std::min<int64_t>(256 * fill / tiles, slices * t.bk / 256);
      if (fill > 0 && want < 2) continue;
      const int per = slices ? ceil_div(slices, want) : 0, splits = slices ? ceil_div(slices, per) : 1;
      if (tiles * splits >= ((int64_t)1 << 32) / t.threads) continue;  // a grid holds fewer than 2^32 threads
      const double us = tiles_us(tile, tiles * splits, per * t.bk / 64.0 * slower) + splits_us(m, n, splits) + (any ? 0 : copies.us);
      if (best != 0 && us >= best) continue;
      best = us;
      p->tile = tile;
      g.slices = slices;
      g.per_split = per;
      g.splits = splits;
      g.tiles_m = (int32_t)tm;
      g.tiles_n = (int32_t)tn;
    }
  }
  if (best == 0)  // 2^23 tiles of 256 x 256 or more: no device has memory for so large an output
    return fail(MUON_EINVAL, "a product of %lld x %lld is too large", (long long)m, (long long)n);
  return MUON_OK;
}

// sizes_only: pointers may be anything (the size of the workspace is asked for), and only
// the distances that its size goes by are checked.
int plan_layer(const muon_linear_t* l, bool backward, void* workspace, bool sizes_only, LinPlan* p) {
  *p = LinPlan{};
  int rc;
  if (!l) return fail(MUON_EINVAL, "arguments are NULL");
  if ((rc = check_dim(l->m, 0, MAX_ROWS, "m")) || (rc = check_dim(l->k, 1, MAX_WIDTH, "k")) ||
      (rc = check_dim(l->n, 1, MAX_WIDTH, "n")))
    return rc;
  if (l->w_transposed != 0 && l->w_transposed != 1) return fail(MUON_EINVAL, "w_transposed = %d is not 0 or 1", l->w_transposed);
  if ((rc = check_epilogue(l->act, l->dropout, l->rng))) return rc;
  const int64_t in = backward ? l->n : l->k, out = backward ? l->k : l->n;  // widths of x and y
  const int type = l->x_type;
  if (type != MUON_BF16 && type != MUON_FP16) return fail(MUON_EINVAL, "x_type = %d: the products take MUON_BF16 and MUON_FP16", type);
  if (l->w_type != type && l->w_type != MUON_FP32) return fail(MUON_EINVAL, "w_type = %d is neither x_type nor MUON_FP32", l->w_type);
  if (l->y_type != type && l->y_type != MUON_FP32) return fail(MUON_EINVAL, "y_type = %d is neither x_type nor MUON_FP32", l->y_type);
  if (l->bias && l->bias_type != type && l->bias_type != MUON_FP32)
    return fail(MUON_EINVAL, "bias_type = %d is neither x_type nor MUON_FP32", l->bias_type);
  if (backward && l->bias) return fail(MUON_EINVAL, "the gradient of the input takes no bias");
  if (backward && (l->act != MUON_ACT_NONE) != (l->preact != nullptr))
    return fail(MUON_EINVAL, "act and preact of the layer below come together");
  p->type = type;
  if (l->m == 0) {
    p->empty = true;
    return MUON_OK;
  }
  const Matrix y = {"y", l->y, l->m, out, l->ldy, l->y_type, true};
  const Matrix x = {"x", l->x, l->m, in, l->ldx, type, false};
  const int64_t w_rows = l->w_transposed ? l->n : l->k, w_cols = l->w_transposed ? l->k : l->n;
  const Matrix w = {"w", l->w, w_rows, w_cols, l->ldw, l->w_type, false};
  if (sizes_only) {
    if ((rc = check_matrix(x, true)) || (rc = check_matrix(w, true))) return rc;
  } else {
    Matrix all[6] = {y, x, w};
    bool may_be_y[6] = {};
    int n = 3;
    if (l->bias) all[n++] = {"bias", l->bias, 1, out, out, l->bias_type, false};
    if (l->preact) {
      may_be_y[n] = backward;
      all[n++] = {"preact", l->preact, l->m, out, l->ldp, type, !backward};
    }
    if (l->residual) {
      may_be_y[n] = true;
      all[n++] = {"residual", l->residual, l->m, out, l->ldr, l->y_type, false};
    }
    for (int i = 0; i < n; ++i)
      if ((rc = check_matrix(all[i]))) return rc;
    if ((rc = check_overlaps(all, may_be_y, n))) return rc;
    if (l->rng && l->dropout > 0.0f) {
      const Matrix rng = {"rng", l->rng, 1, 4, 4, MUON_FP32, false};
      for (int i = 0; i < n; ++i)
        if (all[i].written && overlap(all[i], rng)) return fail(MUON_EINVAL, "%s overlaps rng", all[i].what);
    }
  }
  if ((rc = lay_out(p, l->m, out, in, false, Copies(x, w, type)))) return rc;
  p->b_wide = p->tile == LIN_TILE_64_ANY && w.type == MUON_FP32;
  LinGemmArgs& g = p->gemm;
  g.a = operand_of(x, type, p, workspace);
  g.b = operand_of(w, type, p, workspace);
  // the reduced index runs along w's rows where it is the one they run along
  p->b_kmajor = (l->w_transposed != 0) == backward;
  LinEpilogue& e = g.e;
  e.bias = l->bias;
  e.bias_type = l->bias_type;
  e.residual = l->residual;
  e.ldr = l->ldr;
  e.y = l->y;
  e.ldy = l->ldy;
  e.y_type = l->y_type;
  e.preact = l->preact;
  e.ldp = l->ldp;
  e.act = l->act;
  e.backward = backward;
  fill_dropout(&e, l->dropout, l->seed, l->step, l->site, l->rng);
  if (g.splits > 1) {
    const LinTileSize t = kLinTile[p->tile];
    LinJoinArgs& j = p->join;
    p->finish = true;
    j.part_ld = (int64_t)g.tiles_n * t.bn;
    j.part_stride = j.part_ld * g.tiles_m * t.bm;
    g.part = (float*)take(p, workspace, (size_t)(j.part_stride * g.splits * 4));
    j.part = g.part;
    j.m = g.m;
    j.n = g.n;
    j.splits = g.splits;
    j.e = e;
  }
  return MUON_OK;
}

int plan_grad(const muon_linear_dw_t* l, void* workspace, bool sizes_only, LinPlan* p) {
  *p = LinPlan{};
  int rc;
  if (!l) return fail(MUON_EINVAL, "arguments are NULL");
  if ((rc = check_dim(l->m, 0, MAX_ROWS, "m")) || (rc = check_dim(l->k, 1, MAX_WIDTH, "k")) ||
      (rc = check_dim(l->n, 1, MAX_WIDTH, "n")))
    return rc;
  if (l->dw_transposed != 0 && l->dw_transposed != 1) return fail(MUON_EINVAL, "dw_transposed = %d is not 0 or 1", l->dw_transposed);
  if (l->accumulate != 0 && l->accumulate != 1) return fail(MUON_EINVAL, "accumulate = %d is not 0 or 1", l->accumulate);
  const int type = l->type;
  if (type != MUON_BF16 && type != MUON_FP16) return fail(MUON_EINVAL, "type = %d: the products take MUON_BF16 and MUON_FP16", type);
  p->type = type;
  const int64_t rows = l->dw_transposed ? l->n : l->k, cols = l->dw_transposed ? l->k : l->n;
  const Matrix dw = {"dw", l->dw, rows, cols, l->lddw, MUON_FP32, true};
  const Matrix x = {"x", l->x, l->m, l->k, l->ldx, type, false};
  const Matrix dz = {"dz", l->dz, l->m, l->n, l->lddz, type, false};
  if (sizes_only) {
    if (l->m > 0 && ((rc = check_matrix(x, true)) || (rc = check_matrix(dz, true)))) return rc;
  } else {
    Matrix all[4] = {dw};
    const bool none[4] = {};
    int n = 1;
    if (l->dbias) all[n++] = {"dbias", l->dbias, 1, l->n, l->n, MUON_FP32, true};
    if (l->m > 0) {
      all[n++] = x;
      all[n++] = dz;
    }
    for (int i = 0; i < n; ++i)
      if ((rc = check_matrix(all[i]))) return rc;
    if ((rc = check_overlaps(all, none, n))) return rc;
  }
  p->empty = l->m == 0 && l->accumulate;
  if ((rc = lay_out(p, rows, cols, l->m, true, Copies(x, dz, type)))) return rc;
  LinGemmArgs& g = p->gemm;
  if (l->m > 0) {
    const LinOperand ox = operand_of(x, type, p, workspace), oz = operand_of(dz, type, p, workspace);
    g.a = l->dw_transposed ? oz : ox;
    g.b = l->dw_transposed ? ox : oz;
  }
  g.c = l->dw;
  g.ldc = l->lddw;
  g.add = l->accumulate;
  g.sums = l->dbias;
  g.sum_side = !l->dbias ? 0 : l->dw_transposed ? 2 : 1;
  if (g.splits > 1) {
    const LinTileSize t = kLinTile[p->tile];
    LinFinishArgs& f = p->fin;
    p->finish = true;
    f.part_ld = (int64_t)g.tiles_n * t.bn;
    f.part_stride = f.part_ld * g.tiles_m * t.bm;
    g.part = (float*)take(p, workspace, (size_t)(f.part_stride * g.splits * 4));
    f.c = g.c;
    f.ldc = g.ldc;
    f.add = g.add;
    f.part = g.part;
    f.m = g.m;
    f.n = g.n;
    f.splits = g.splits;
    f.sum_first_block = ceil_div((int64_t)g.m * ((g.n + 7) / 8), FINISH_THREADS);
    if (g.sum_side) {
      f.sums = g.sums;
      f.n_sums = (int32_t)l->n;
      f.sum_rows = g.splits * (g.sum_side == 1 ? g.tiles_m : g.tiles_n);
      f.sum_stride = g.sum_side == 1 ? f.part_ld : (int64_t)g.tiles_m * t.bm;
      g.sum_part = (float*)take(p, workspace, (size_t)(f.sum_stride * f.sum_rows * 4));
      f.sum_part = g.sum_part;
    }
  }
  return MUON_OK;
}

// The workspace as the caller gave it.
int check_workspace(const LinPlan& p, const void* workspace, size_t bytes) {
  if (p.empty || p.workspace == 0) return MUON_OK;
  if (!workspace) return fail(MUON_EINVAL, "workspace is NULL; this call needs %zu bytes", p.workspace);
  if ((uintptr_t)workspace % 16) return fail(MUON_EINVAL, "workspace is not 16-byte aligned");
  if (bytes < p.workspace) return fail(MUON_ENOMEM, "workspace of %zu bytes; this call needs %zu", bytes, p.workspace);
  return MUON_OK;
}

int check_workspace_apart(const LinPlan& p, const void* workspace, const Matrix* m, int n) {
  if (p.empty || p.workspace == 0) return MUON_OK;
  const Matrix ws = {"workspace", workspace, 1, (int64_t)(p.workspace / 4), (int64_t)(p.workspace / 4), MUON_FP32, true};
  for (int i = 0; i < n; ++i)
    if (m[i].p && m[i].rows > 0 && m[i].lo() < ws.hi() && ws.lo() < m[i].hi())
      return fail(MUON_EINVAL, "workspace overlaps %s", m[i].what);
  return MUON_OK;
}

}  // namespace

int plan_linear(const muon_linear_t* l, bool backward, void* workspace, size_t workspace_bytes, LinPlan* out) {
  int rc = plan_layer(l, backward, workspace, false, out);
  if (rc || (rc = check_workspace(*out, workspace, workspace_bytes)) || out->empty) return rc;
  const int64_t in = backward ? l->n : l->k, to = backward ? l->k : l->n;
  const Matrix all[] = {{"y", l->y, l->m, to, l->ldy, l->y_type, true},
                        {"x", l->x, l->m, in, l->ldx, l->x_type, false},
                        {"w", l->w, l->w_transposed ? l->n : l->k, l->w_transposed ? l->k : l->n, l->ldw, l->w_type, false},
                        {"bias", l->bias, 1, to, to, l->bias_type, false},
                        {"preact", l->preact, l->m, to, l->ldp, l->x_type, !backward},
                        {"residual", l->residual, l->m, to, l->ldr, l->y_type, false},
                        {"rng", l->rng, 1, 4, 4, MUON_FP32, false}};
  return check_workspace_apart(*out, workspace, all, 7);
}

int plan_linear_dw(const muon_linear_dw_t* l, void* workspace, size_t workspace_bytes, LinPlan* out) {
  int rc = plan_grad(l, workspace, false, out);
  if (rc || (rc = check_workspace(*out, workspace, workspace_bytes)) || out->empty) return rc;
  const Matrix all[] = {{"dw", l->dw, l->dw_transposed ? l->n : l->k, l->dw_transposed ? l->k : l->n, l->lddw, MUON_FP32, true},
                        {"dbias", l->dbias, 1, l->n, l->n, MUON_FP32, true},
                        {"x", l->x, l->m, l->k, l->ldx, l->type, false},
                        {"dz", l->dz, l->m, l->n, l->lddz, l->type, false}};
  return check_workspace_apart(*out, workspace, all, 4);
}

int linear_workspace(const muon_linear_t* l, bool backward, size_t* bytes) {
  LinPlan p;
  const int rc = plan_layer(l, backward, nullptr, true, &p);
  *bytes = rc ? 0 : p.workspace;
  return rc;
}

int linear_dw_workspace(const muon_linear_dw_t* l, size_t* bytes) {
  LinPlan p;
  const int rc = plan_grad(l, nullptr, true, &p);
  *bytes = rc ? 0 : p.workspace;
  return rc;
}

int plan_dropout(const muon_dropout_t* d, DropArgs* out, int64_t* blocks) {
  *out = DropArgs{};
  *blocks = 0;
  int rc;
  if (!d) return fail(MUON_EINVAL, "arguments are NULL");
  if ((rc = check_dim(d->m, 0, MAX_ROWS, "m")) || (rc = check_dim(d->n, 0, MUON_DROPOUT_MAX_COLS, "n"))) return rc;
  if ((rc = check_epilogue(d->act, d->dropout, d->rng))) return rc;
  if ((d->act != MUON_ACT_NONE) != (d->preact != nullptr)) return fail(MUON_EINVAL, "act and preact come together");
  if (d->x_type < MUON_FP32 || d->x_type > MUON_FP16) return fail(MUON_EINVAL, "x_type = %d is no element type", d->x_type);
  if (d->y_type < MUON_FP32 || d->y_type > MUON_FP16) return fail(MUON_EINVAL, "y_type = %d is no element type", d->y_type);
  if (d->m == 0 || d->n == 0) return MUON_OK;
  Matrix all[4] = {{"y", d->y, d->m, d->n, d->ldy, d->y_type, true}, {"x", d->x, d->m, d->n, d->ldx, d->x_type, false}};
  const bool may_be_y[4] = {false, true, true, true};
  int n = 2;
  if (d->preact) all[n++] = {"preact", d->preact, d->m, d->n, d->ldp, d->x_type, false};
  if (d->residual) all[n++] = {"residual", d->residual, d->m, d->n, d->ldr, d->y_type, false};
  for (int i = 0; i < n; ++i)
    if ((rc = check_matrix(all[i]))) return rc;
  if ((rc = check_overlaps(all, may_be_y, n))) return rc;
  if (d->rng && d->dropout > 0.0f && overlap(all[0], Matrix{"rng", d->rng, 1, 4, 4, MUON_FP32, false}))
    return fail(MUON_EINVAL, "y overlaps rng");
  const int64_t eights = d->m * ((d->n + 7) / 8);
  *blocks = (eights + DROP_THREADS - 1) / DROP_THREADS;
  if (*blocks > MAX_LAUNCH_ITEMS) return fail(MUON_EINVAL, "%lld x %lld elements are too many", (long long)d->m, (long long)d->n);
  out->x = d->x;
  out->ldx = d->ldx;
  out->m = d->m;
  out->n = d->n;
  out->x_type = d->x_type;
  LinEpilogue& e = out->e;
  e.residual = d->residual;
  e.ldr = d->ldr;
  e.y = d->y;
  e.ldy = d->ldy;
  e.y_type = d->y_type;
  e.preact = const_cast<void*>(d->preact);
  e.ldp = d->ldp;
  e.act = d->act;
  e.backward = 1;
  fill_dropout(&e, d->dropout, d->seed, d->step, d->site, d->rng);
  return MUON_OK;
}

}  // namespace muon
