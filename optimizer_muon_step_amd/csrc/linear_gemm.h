// Matrix products of a layer's forward and backward pass on gfx950 matrix
// cores: C = A B over 16-bit operands, sums in fp32.
//
//   forward  y = x w        A = x, rows of k        B = w, rows of n, or of k
//   dx       dz w^T         A = dz, rows of n       B = w^T, likewise
//   dw       x^T dz         A = x^T and B = dz, both rows of the other index
//
// An operand is k-contiguous (its rows run along the reduced index) or k-major
// (its rows run along the output's index), so that no layout has to be
// transposed in memory: k-major slices go through the transposing LDS read.
//
// Pipeline: WM x WN x WK waves over a BM x BN tile.  K advances in slices of
// 64 through a ring of NSTAGE LDS buffers that buffer loads fill directly (no
// registers), every row segment a whole 128-byte line.  Buffer loads bound every access by the
// operand's own end and give zeros behind it, which serves the rows and
// columns that a tile hangs over and the rows behind K; the chunks behind K
// of k-contiguous rows, where the next row follows, get an offset that is
// out of bounds by itself.  The 16-byte chunks are XOR-swizzled on the
// global side, since each lane's LDS slot is fixed by its lane id.
// WK > 1 gives the k-steps of a slice to WK groups of waves whose sums meet in LDS at the end: a
// small tile then has enough waves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_epilogue.h"

namespace muon {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
#define LIN_LDS __attribute__((address_space(3)))

// Wait until at most n vector-memory operations of this wave are outstanding,
// and all of its LDS operations are done (gfx9 encoding of s_waitcnt).
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "beyond the counter");
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4));
}
// At most `after` slices of PER loads each, `after` below NSTAGE - 1.
template <int PER, int NSTAGE>
__device__ __forceinline__ void wait_slices(int after) {
  if (NSTAGE > 7 && after >= 6) wait_loads<6 * PER>();
  else if (NSTAGE > 6 && after == 5) wait_loads<5 * PER>();
  else if (NSTAGE > 5 && after == 4) wait_loads<4 * PER>();
  else if (NSTAGE > 4 && after == 3) wait_loads<3 * PER>();
  else if (NSTAGE > 3 && after == 2) wait_loads<2 * PER>();
  else if (NSTAGE > 2 && after == 1) wait_loads<PER>();
  else wait_loads<0>();
}

__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 bytes a lane from a buffer to LDS at `to` + 16 lane.  Written out, since
// before every LDS read the compiler would wait for all of its own such loads,
// those of later slices among them; the waits are wait_loads'.  It has no
// result in registers, and nothing else in these kernels uses M0.  M0 has to be
// set one wait state ahead, and a descriptor that a vector instruction left
// (`fresh`) five.
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t to, uint32_t off, bool fresh) {
  if (fresh)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(rsrc) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(rsrc) : "memory");
}

template <int TYPE>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (TYPE == GRAD_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// One operand's slice in LDS: R rows (k-contiguous, 128 bytes each) or 64
// rows of R elements (k-major), the loads that fill it and the fragment reads.
template <bool KMAJOR, int R, int NW>
struct Slice {
  static constexpr int BYTES = R * LIN_BK * 2;
  static constexpr int LOADS = R / 8 / NW;   // 1 KB each, per wave
  static constexpr int CHUNKS = KMAJOR ? R / 8 : LIN_BK / 8;  // 16-byte chunks of a row
  static constexpr int ROWS = 64 / CHUNKS;   // rows of one load
  static_assert(R % 32 == 0 && LOADS >= 1 && LOADS * 8 * NW == R, "tile does not split into whole loads");
  static_assert(!KMAJOR || R == 64 || R == 128 || R == 256, "k-major rows of 128, 256 or 512 bytes");

  // Chunk swizzle.  A k-contiguous fragment has 16 lanes on 16 rows at
  // one chunk; two rows share a 256-byte line of the banks, so XOR by (row / 2) % 8
  // puts the 16 reads on 16 chunks.  A transposing read has each 16 lanes on 4
  // rows, 32 bytes each, and pairs of such groups 32 bytes apart; the XOR sends the
  // 4 rows to different 64-byte groups of the banks.
  static __device__ __forceinline__ int swz(int row, int chunk) {
    if (!KMAJOR) return chunk ^ ((row >> 1) & 7);
    return CHUNKS == 8 ? chunk ^ (4 * ((row >> 1) & 1)) : chunk ^ (4 * (row & 3));
  }

  uint64_t base;     // of the slice that is loaded next
  int64_t left;      // bytes from there to the operand's end
  int64_t step;      // from slice to slice
  uint32_t vo[LOADS];  // this lane's offsets within a slice

  // Of the tile that starts at row / column `first`, from slice s0 on.
  __device__ __forceinline__ void start(const LinOperand& o, int first, int s0, int wave, int lane) {
    step = KMAJOR ? LIN_BK * o.ld : LIN_BK * 2;
    const int64_t at = (KMAJOR ? (int64_t)first * 2 : (int64_t)first * o.ld) + s0 * step;
    base = (uint64_t)o.p + at;
    left = o.bytes - at;
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      const int row = (t * NW + wave) * ROWS + lane / CHUNKS;
      vo[t] = (uint32_t)(row * (int)o.ld) + swz(row, lane % CHUNKS) * 16;
    }
  }

  // The next slice into LDS at `to`.  have: elements of K from the slice's start.
  __device__ __forceinline__ void load(LIN_LDS char* to, int have, int wave, int lane) {
    // offsets stay below 2^31 - 16, and so do the records: an offset of 2^31 is out of bounds
    const int records = (int)min(left, (int64_t)0x7ffffff0);
    const i32x4 rsrc = {(int)(uint32_t)base, (int)(uint32_t)(base >> 32) & 0xffff, records, 0x00020000};
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      uint32_t off = vo[t];
      if (!KMAJOR && have < LIN_BK) {  // have is a multiple of 8
        const int row = (t * NW + wave) * ROWS + lane / CHUNKS;
        if (swz(row, lane % CHUNKS) * 8 >= have) off = 0x80000000u;
      }
      load_to_lds(rsrc, (uint32_t)(uintptr_t)(to + (t * NW + wave) * 1024), off, t == 0);
    }
    base += step;
    left -= step;
  }

  // Offsets within the slice of this lane's reads of the 32 x 16 fragment at
  // row / column r0, k-step 0.
  struct Read {
    int lo, hi;
  };
  static __device__ __forceinline__ Read read_of(int r0, int lane) {
    if (!KMAJOR) {
      const int r = r0 + (lane & 31);
      return {r * 128 + swz(r, lane >> 5) * 16, 0};
    }
    // ds_read_b64_tr_b16 transposes 16-bit elements across 16 lanes: with lane L
    // of a group addressing row k0 + L/4, columns j0 + 4(L%4) .. +3, lane i
    // receives column j0 + i of rows k0 .. k0+3
    const int g = lane >> 4, l = lane & 15;
    const int k = 8 * (g >> 1) + (l >> 2), j = r0 + 16 * (g & 1) + 4 * (l & 3);
    return {k * (2 * R) + swz(k, j >> 3) * 16 + (j & 7) * 2, (k + 4) * (2 * R) + swz(k + 4, j >> 3) * 16 + (j & 7) * 2};
  }
  // Element i of a lane: row / column r0 + lane % 32, k = 16 kk + 8 (lane / 32) + i.
  static __device__ __forceinline__ s16x8 fragment(const LIN_LDS char* st, Read r, int kk) {
    if (!KMAJOR) return *(const LIN_LDS s16x8*)(st + (r.lo ^ (32 * kk)));  // chunk 2 kk further on: an XOR too
    // 16 rows on: the swizzle is the same
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LIN_LDS s16x4*)(st + r.lo + kk * 16 * (2 * R)));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LIN_LDS s16x4*)(st + r.hi + kk * 16 * (2 * R)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

template <int TYPE>
__device__ __forceinline__ float fragment_sum(s16x8 f) {
  const f32x8 v = widen8<TYPE>(__builtin_bit_cast(u32x4, f));
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// What a tile's sums become: eight of them at (row, col ..), or one.
template <int TYPE>
struct LayerStore {
  const LinEpilogue& e;
  const DropKey key;
  __device__ __forceinline__ explicit LayerStore(const LinGemmArgs& a) : e(a.e), key(a.e) {}

  static __device__ __forceinline__ f32x8 get(int type, const void* p, int64_t i) {
    return type == GRAD_FP32 ? load8<GRAD_FP32>(p, i) : load8<TYPE>(p, i);
  }
  static __device__ __forceinline__ float get1(int type, const void* p, int64_t i) {
    return type == GRAD_FP32 ? load1<GRAD_FP32>(p, i) : load1<TYPE>(p, i);
  }

  __device__ __forceinline__ void operator()(int64_t row, int col, f32x8 v) const {
    if (!e.backward) {
      if (e.bias) v += get(e.bias_type, e.bias, col);
      if (e.preact) store8<TYPE>(e.preact, row * e.ldp + col, v);
      if (e.act != LIN_ACT_NONE) v = act8(v, e.act);
    } else if (e.act != LIN_ACT_NONE) {
      v = slope8(load8<TYPE>(e.preact, row * e.ldp + col), e.act) * v;
    }
    if (e.border != 0) v = drop8(e, key, row, col, v);
    if (e.residual) v = get(e.y_type, e.residual, row * e.ldr + col) + v;
    if (e.y_type == GRAD_FP32) store8<GRAD_FP32>(e.y, row * e.ldy + col, v);
    else store8<TYPE>(e.y, row * e.ldy + col, v);
  }
  __device__ __forceinline__ void one(int64_t row, int col, float v) const {
    if (!e.backward) {
      if (e.bias) v += get1(e.bias_type, e.bias, col);
      if (e.preact) store1<TYPE>(e.preact, row * e.ldp + col, v);
      v = act_of(v, e.act);
    } else if (e.act != LIN_ACT_NONE) {
      v *= act_slope(load1<TYPE>(e.preact, row * e.ldp + col), e.act);
    }
    if (e.border != 0) v = drop1(e, key, row, col, v);
    if (e.residual) v = get1(e.y_type, e.residual, row * e.ldr + col) + v;
    if (e.y_type == GRAD_FP32) store1<GRAD_FP32>(e.y, row * e.ldy + col, v);
    else store1<TYPE>(e.y, row * e.ldy + col, v);
  }
};

struct GradStore {
  float* c;
  int64_t ldc;
  bool add;
  __device__ __forceinline__ void operator()(int64_t row, int col, f32x8 v) const {
    if (add) v = load8<GRAD_FP32>(c, row * ldc + col) + v;
    store8<GRAD_FP32>(c, row * ldc + col, v);
  }
  __device__ __forceinline__ void one(int64_t row, int col, float v) const {
    if (add) v = load1<GRAD_FP32>(c, row * ldc + col) + v;
    store1<GRAD_FP32>(c, row * ldc + col, v);
  }
};

template <int TYPE, bool AK, bool BK, bool GRAD, int BM, int BN, int WM, int WN, int WK, int NSTAGE>
__global__ __launch_bounds__(64 * WM * WN * WK) void linear_gemm_kernel(const LinGemmArgs a) {
  constexpr int NW = WM * WN * WK;
  constexpr int WTM = BM / WM, WTN = BN / WN;  // wave tile
  constexpr int TM = WTM / 32, TN = WTN / 32;
  typedef Slice<AK, BM, NW> SA;
  typedef Slice<BK, BN, NW> SB;
  constexpr int STAGE = SA::BYTES + SB::BYTES;
  constexpr int PER = SA::LOADS + SB::LOADS;
  constexpr int STEPS = LIN_BK / 16;
  constexpr int PITCH = WTN * 4 + 16;  // staged fp32 rows: 16 bytes more move each row to other banks
  constexpr int STAGED = NW * 32 * PITCH;
  constexpr int LDS = NSTAGE * STAGE > STAGED ? NSTAGE * STAGE : STAGED;
  static_assert(NSTAGE >= 2 && NSTAGE <= 8 && (NSTAGE - 2) * PER < 64 && LDS <= 160 * 1024, "ring");
  static_assert(STEPS % WK == 0 && TM * 32 == WTM && TN * 32 == WTN, "wave tile");
  __shared__ __attribute__((aligned(16))) char lds[LDS];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave / (WM * WN), wi = wave / WN % WM, wj = wave % WN;

  // The block's tile.
  const int tiles = a.tiles_m * a.tiles_n, items = tiles * a.splits;
  const int xcd = blockIdx.x & 7, run = items >> 3, longer = items & 7;
  const int item = xcd * run + min(xcd, longer) + (blockIdx.x >> 3);
  const int split = item / tiles, tile = item - split * tiles;
  const int group = tile / (LIN_GROUP * a.tiles_n), in_group = tile - group * LIN_GROUP * a.tiles_n;
  const int gm = min(LIN_GROUP, a.tiles_m - group * LIN_GROUP);
  const int tn = in_group / gm, tm = group * LIN_GROUP + in_group - tn * gm;
  const int row0 = tm * BM, col0 = tn * BN;
  const int s0 = split * a.per_split, slices = min(a.per_split, a.slices - s0);

  SA la;
  SB lb;
  la.start(a.a, row0, s0, wave, lane);
  lb.start(a.b, col0, s0, wave, lane);
  auto stage_of = [&](int s) { return (LIN_LDS char*)lds + (s % NSTAGE) * STAGE; };
  auto issue = [&](int s) {
    const int have = a.k - (s0 + s) * LIN_BK;
    la.load(stage_of(s), have, wave, lane);
    lb.load(stage_of(s) + SA::BYTES, have, wave, lane);
  };

  typename SA::Read ra[TM];
  typename SB::Read rb[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) ra[i] = SA::read_of(wi * WTM + i * 32, lane);
#pragma unroll
  for (int j = 0; j < TN; ++j) rb[j] = SB::read_of(wj * WTN + j * 32, lane);

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = 0.0f;
  // Sums of dz over its rows, of the fragments this wave reads of it: every
  // slice in the first tile across, or with splits the slices shared out over the tiles across.
  constexpr int TS = TM > TN ? TM : TN;
  float sum[GRAD ? TS : 1] = {};
  const int across = GRAD ? (a.sum_side == 1 ? tm : tn) : 0;
  const int sharers = GRAD && a.splits > 1 ? (a.sum_side == 1 ? a.tiles_m : a.tiles_n) : 1;
  const bool summing = GRAD && ((a.sum_side == 1 && wi == 0) || (a.sum_side == 2 && wj == 0)) && (a.splits > 1 || across == 0);

  auto compute = [&](int s) {
    const LIN_LDS char* sa = stage_of(s);
    const LIN_LDS char* sb = sa + SA::BYTES;
#pragma unroll
    for (int t = 0; t < STEPS / WK; ++t) {
      const int kk = WK == 1 ? t : t * WK + wk;
      s16x8 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = SA::fragment(sa, ra[i], kk);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = SB::fragment(sb, rb[j], kk);
      // operands swapped: a lane then holds 4 consecutive columns of one row
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma<TYPE>(fb[j], fa[i], acc[i][j]);
    }
    if constexpr (GRAD) {
      if (summing && (sharers == 1 || (s0 + s) % sharers == across)) {
#pragma unroll
        for (int t = 0; t < STEPS / WK; ++t) {
          const int kk = WK == 1 ? t : t * WK + wk;
          if (a.sum_side == 1) {
#pragma unroll
            for (int j = 0; j < TN; ++j) sum[j] += fragment_sum<TYPE>(SB::fragment(sb, rb[j], kk));
          } else {
#pragma unroll
            for (int i = 0; i < TM; ++i) sum[i] += fragment_sum<TYPE>(SA::fragment(sa, ra[i], kk));
          }
        }
      }
    }
  };

  // Slice s is there once this wave has only the loads of later slices
  // outstanding and every wave has passed the barrier; the buffer that is filled next
  // was last read in step s - 1, which every wave had finished (its LDS reads
  // included) before the barrier.
#pragma unroll
  for (int s = 0; s < NSTAGE - 1; ++s)
    if (s < slices) issue(s);
  for (int s = 0; s < slices; ++s) {
    wait_slices<PER, NSTAGE>(min(NSTAGE - 2, slices - 1 - s));
    block_barrier();
    if (s + NSTAGE - 1 < slices) issue(s + NSTAGE - 1);
    compute(s);
  }
  wait_loads<0>();
  block_barrier();

  // The sums go through LDS, 32 rows of each wave at a time, and are stored in
  // eights of consecutive columns, whole lines of the output.
  LIN_LDS char* staged = (LIN_LDS char*)lds + wave * (32 * PITCH);
  LIN_LDS char* first = (LIN_LDS char*)lds + (wave % (WM * WN)) * (32 * PITCH);  // of the wave tile's group wk = 0
  constexpr int EIGHTS = WTN / 8;
  const bool to_part = GRAD && a.splits > 1;
  const int rows = to_part ? a.tiles_m * BM : a.m, cols = to_part ? a.tiles_n * BN : a.n;
  auto stored = [&](auto&& store) {
#pragma unroll 1
    for (int i = 0; i < TM; ++i) {
      f32x16 v[TN];
#pragma unroll
      for (int q = 0; q < TM; ++q)
        if (q == i) {
#pragma unroll
          for (int j = 0; j < TN; ++j) v[j] = acc[q][j];
        }
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *(LIN_LDS f32x4*)(staged + (lane & 31) * PITCH + (j * 32 + 8 * e + 4 * (lane >> 5)) * 4) =
              f32x4{v[j][4 * e], v[j][4 * e + 1], v[j][4 * e + 2], v[j][4 * e + 3]};
      wait_loads<63>();  // LDS only
      if (WK > 1) block_barrier(); else asm volatile("" ::: "memory");
#pragma unroll
      for (int t = 0; t < 32 * EIGHTS / (64 * WK); ++t) {
        const int q = (t * WK + wk) * 64 + lane, r = q / EIGHTS, c = q % EIGHTS;
        const LIN_LDS char* at = first + r * PITCH + c * 32;
        const int row = row0 + wi * WTM + i * 32 + r, col = col0 + wj * WTN + c * 8;
        if (row >= rows) continue;
        if (col + 8 <= cols) {
          f32x8 x = 0.0f;
#pragma unroll
          for (int w = 0; w < WK; ++w) {
            const LIN_LDS char* p = at + w * (WM * WN * 32 * PITCH);
            const f32x4 lo = *(const LIN_LDS f32x4*)p, hi = *(const LIN_LDS f32x4*)(p + 16);
            const f32x8 y = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            x = w == 0 ? y : x + y;
          }
          store(row, col, x);
        } else {  // the last columns, one by one
#pragma unroll 1
          for (int k = 0; col + k < cols; ++k) {
            float x = *(const LIN_LDS float*)(at + 4 * k);
#pragma unroll
            for (int w = 1; w < WK; ++w) x += *(const LIN_LDS float*)(at + 4 * k + w * (WM * WN * 32 * PITCH));
            store.one(row, col + k, x);
          }
        }
      }
      wait_loads<63>();
      if (WK > 1) block_barrier(); else asm volatile("" ::: "memory");
    }
  };
  if constexpr (!GRAD) {
    stored(LayerStore<TYPE>(a));
  } else {
    if (to_part) {
      const int64_t ld = (int64_t)a.tiles_n * BN;
      stored(GradStore{a.part + split * (ld * a.tiles_m * BM), ld, false});
    } else {
      stored(GradStore{a.c, a.ldc, a.add != 0});
    }
    if (a.sum_side != 0) {
      const int edge = a.sum_side == 1 ? BN : BM, wt = a.sum_side == 1 ? WTN : WTM, frags = wt / 32;
      LIN_LDS float* red = (LIN_LDS float*)lds;  // WK x edge
      block_barrier();
      if (summing) {
#pragma unroll
        for (int f = 0; f < TS; ++f) {
          if (f >= frags) break;
          const float v = sum[f] + __shfl_xor(sum[f], 32);
          if (lane < 32) red[wk * edge + (a.sum_side == 1 ? wj : wi) * wt + f * 32 + lane] = v;
        }
      }
      wait_loads<63>();
      block_barrier();
      if (to_part || across == 0) {
        const int at = (a.sum_side == 1 ? col0 : row0), limit = a.sum_side == 1 ? a.n : a.m;
        const int64_t width = (int64_t)(a.sum_side == 1 ? a.tiles_n : a.tiles_m) * edge;
        for (int t = threadIdx.x; t < edge; t += 64 * NW) {
          float v = red[t];
#pragma unroll
          for (int w = 1; w < WK; ++w) v += red[w * edge + t];
          if (to_part) gptr(a.sum_part)[(split * (int64_t)sharers + across) * width + at + t] = v;
          else if (at + t < limit) gptr(a.sums)[at + t] = a.add ? gptr(a.sums)[at + t] + v : v;
        }
      }
    }
  }
}

}  // namespace lin
}  // namespace muon
