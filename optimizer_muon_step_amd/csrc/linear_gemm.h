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
// BK through a ring of NSTAGE LDS buffers that buffer loads fill directly (no
// registers), every row segment whole 128-byte lines.  The fragments of a k-step
// are read while the matrix cores work on the step before, across the slices'
// borders too: the barrier that hands over the next slice stands before the last
// k-step of the current one.  Buffer loads bound every access by the
// operand's own end and give zeros behind it, which serves the rows and
// columns that a tile hangs over and the rows behind K; the chunks behind K
// of k-contiguous rows, where the next row follows, get an offset that is
// out of bounds by itself.  The 16-byte chunks are XOR-swizzled on the
// global side, since each lane's LDS slot is fixed by its lane id.
// WK > 1 gives the k-steps of a slice to WK groups of waves whose sums meet in LDS at the end: a
// small tile then has enough waves.
//
// Measured (bf16, one MI355X): 16384 x 3072 over 768 with GELU and z kept 102 us, 760
// TFLOP/s, 65 us of it the main loop and the rest 200 MB of stores that a round of tiles
// ends with; 32768 x 6400 over 1600, likewise, 690 us, 970 TFLOP/s, matrix cores busy 43 %: with 256 x 256 tiles
// of 8 waves LDS reads and barriers take their turns beside them (at 8192^3 540 us of matrix instructions alone, 612
// with the reads, 630 with barriers, 800 with the loads).  16384 x 768 over
// 3072 is 256 tiles of 256 x 192, one to a compute unit: 81 us with dropout and residual.  One row of
// 2304 over 768 is latency, 5.4 us.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "linear_epilogue.h"

namespace muon {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
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
  if constexpr (NSTAGE > 2) {
    if (after == NSTAGE - 2) wait_loads<(NSTAGE - 2) * PER>();
    else wait_slices<PER, NSTAGE - 1>(after);
  } else {
    wait_loads<0>();
  }
}

__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 bytes a lane from a buffer to LDS at `to` + 16 lane.  Written out, since
// before every LDS read the compiler would wait for all of its own such loads,
// those of later slices among them; the waits are wait_loads'.  It has no
// result in vector registers.  M0 has to be set one wait state ahead, and a
// descriptor that a vector instruction left (a spilled scalar's way back, too) five.
__device__ __forceinline__ void load_to_lds(i32x4 rsrc, uint32_t to, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(rsrc) : "m0", "memory");
}

template <int TYPE>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (TYPE == GRAD_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// One operand's slice in LDS: R rows of BK elements (k-contiguous) or BK rows
// of R elements (k-major), the loads that fill it and the fragment reads.
template <bool KMAJOR, int R, int NW, int BK>
struct Slice {
  static constexpr int BYTES = R * BK * 2;
  static constexpr int PIECES = BYTES / 1024, LOADS = (PIECES + NW - 1) / NW;  // 1 KB each, per wave
  static constexpr int PITCH = KMAJOR ? R * 2 : BK * 2;  // bytes of a row
  static constexpr int CHUNKS = PITCH / 16;  // 16-byte chunks of a row
  static_assert(R % 32 == 0 && PIECES * 1024 == BYTES && PIECES >= NW, "tile does not split into whole loads");
  static_assert(BK == 128 || BK == 64, "k-contiguous rows of 256 or 128 bytes");
  static_assert(!KMAJOR || R % 64 == 0, "k-major rows of multiples of 128 bytes: the swizzle stays within 8 chunks");

  // Chunk swizzle.  A k-contiguous fragment has 16 lanes on 16 rows at one
  // chunk; a row of 128 elements fills a 256-byte line of the banks and two rows of
  // 64 share one, so XOR by row % 16, or (row / 2) % 8, puts the 16 reads on 16
  // chunks.  A transposing read has each 16 lanes on 4 rows, 32 bytes each, and the
  // next 16 lanes 8 rows further on; the XOR sends the 4 rows to different 64-byte
  // groups of the banks and the 8 rows to the other half of such a group.
  // Piece t of a wave.  Where they do not divide, some waves load the last one too: each
  // has the same number of loads to wait for.
  static __device__ __forceinline__ int piece(int t, int wave) {
    return PIECES % NW == 0 ? t * NW + wave : min(t * NW + wave, PIECES - 1);
  }
  static __device__ __forceinline__ int swz(int row, int chunk) {
    if (!KMAJOR) return BK == 64 ? chunk ^ ((row >> 1) & 7) : chunk ^ (row & 15);
    return chunk ^ (PITCH % 256 != 0 ? 4 * ((row >> 1) & 1) : 4 * (row & 3)) ^ (2 * ((row >> 3) & 1));
  }

  uint64_t base;     // of the slice that is loaded next
  int64_t left;      // bytes from there to the operand's end
  int64_t step;      // from slice to slice
  uint32_t vo[LOADS];  // this lane's offsets within a slice

  // Of the tile that starts at row / column `first`, from slice s0 on.
  __device__ __forceinline__ void start(const LinOperand& o, int first, int s0, int wave, int lane) {
    step = KMAJOR ? BK * o.ld : BK * 2;
    const int64_t at = (KMAJOR ? (int64_t)first * 2 : (int64_t)first * o.ld) + s0 * step;
    base = (uint64_t)o.p + at;
    left = o.bytes - at;
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      const int slot = piece(t, wave) * 64 + lane, row = slot / CHUNKS;
      vo[t] = (uint32_t)(row * (int)o.ld) + swz(row, slot % CHUNKS) * 16;
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
      if (!KMAJOR && have < BK) {  // the chunk that K ends in holds zeros from there on
        const int slot = piece(t, wave) * 64 + lane;
        if (swz(slot / CHUNKS, slot % CHUNKS) * 8 >= have) off = 0x80000000u;
      }
      load_to_lds(rsrc, (uint32_t)(uintptr_t)(to + piece(t, wave) * 1024), off);
    }
    base += step;
    left -= step;
  }

  // Offsets within the slice of this lane's reads of the 16 x 32 fragment at
  // row / column r0, k-step 0.
  struct Read {
    int lo, hi;
  };
  static __device__ __forceinline__ Read read_of(int r0, int lane) {
    const int g = lane >> 4, l = lane & 15;
    if (!KMAJOR) {
      const int r = r0 + l;
      return {r * PITCH + swz(r, g) * 16, 0};
    }
    // ds_read_b64_tr_b16 transposes 16-bit elements across 16 lanes: with lane L
    // of a group addressing row k0 + L/4, columns j0 + 4(L%4) .. +3, lane i
    // receives column j0 + i of rows k0 .. k0+3
    const int k = 8 * g + (l >> 2), j = r0 + 4 * (l & 3);
    return {k * PITCH + swz(k, j >> 3) * 16 + (j & 7) * 2, (k + 4) * PITCH + swz(k + 4, j >> 3) * 16 + (j & 7) * 2};
  }
  // Element i of a lane: row / column r0 + lane % 16, k = 32 kk + 8 (lane / 16) + i.
  static __device__ __forceinline__ s16x8 fragment(const LIN_LDS char* st, Read r, int kk) {
    if (!KMAJOR) return *(const LIN_LDS s16x8*)(st + (r.lo ^ (64 * kk)));  // chunk 4 kk further on: an XOR too
    // 32 rows on: the swizzle is the same
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LIN_LDS s16x4*)(st + r.lo + kk * 32 * PITCH));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LIN_LDS s16x4*)(st + r.hi + kk * 32 * PITCH));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

// The same slice through registers, of an operand that buffer loads to LDS cannot
// read: rows that start at any element, of any length from 8 on, of 16 or (WIDE)
// 32 bits, the latter rounded to TYPE on the way.  Every load is of 8 elements within the operand: a chunk
// that its row ends in is read from 8 before the row's end on and moved down, one
// outside is read elsewhere.  What lies behind K becomes zeros; rows and columns that
// the tile hangs over hold something, which the output's bounds leave out.  A slice of 128 takes
// about 1.2 times as long as by direct loads, 1.7 times where rows start off 16 bytes; what it saves
// is the copy's launch and its pass (linear_host.cpp weighs them).
template <int TYPE, bool WIDE, bool KMAJOR, int R, int NW, int BK>
struct AnySlice : Slice<KMAJOR, R, NW, BK> {
  typedef Slice<KMAJOR, R, NW, BK> Base;
  using Base::CHUNKS;
  using Base::LOADS;
  static_assert(Base::PIECES % NW == 0, "whole loads");
  using Base::swz;
  static constexpr int SIZE = WIDE ? 4 : 2;
  struct Held {
    u32x4 lo[LOADS], hi[WIDE ? LOADS : 1];
  };

  const char* base;
  int64_t ld;        // bytes
  int rows, cols;    // as stored
  int first;
  int64_t at[LOADS];  // k-contiguous: of this lane's row; k-major: of its columns
  int place[LOADS];   // k-contiguous: the chunk's first column; k-major: its row in a slice
  int down[LOADS];    // k-major: elements to move down

  __device__ __forceinline__ void start(const LinOperand& o, int first_, int side, int k, int wave, int lane) {
    base = (const char*)o.p;
    ld = o.ld;
    first = first_;
    rows = KMAJOR ? k : side;
    cols = KMAJOR ? side : k;
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      const int slot = (t * NW + wave) * 64 + lane, row = slot / CHUNKS, col = swz(row, slot % CHUNKS) * 8;
      if (KMAJOR) {
        const int from = min(first + col, cols - 8);
        at[t] = (int64_t)from * SIZE;
        down[t] = first + col - from;
        place[t] = row;
      } else {
        at[t] = min(first + row, rows - 1) * ld;
        place[t] = col;
      }
    }
  }

  // Slice s of K.
  __device__ __forceinline__ void fetch(Held& h, int s) const {
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      const int p = s * BK + place[t];
      int64_t off;
      if (KMAJOR) off = at[t] + min(p, rows - 1) * ld;
      else off = at[t] + (int64_t)(p + 8 <= cols ? p : p < cols ? cols - 8 : 0) * SIZE;
      const char* from = base + off;
      if (WIDE) {
        h.lo[t] = __builtin_bit_cast(u32x4, load_raw4(from));
        h.hi[t] = __builtin_bit_cast(u32x4, load_raw4(from + 16));
      } else {
        h.lo[t] = load_raw<GRAD_BF16>(from, 0);
      }
    }
  }
  static __device__ __forceinline__ f32x4 load_raw4(const char* p) {
    const f32x4_u w = *reinterpret_cast<const MUON_GLOBAL f32x4_u*>(gptr(reinterpret_cast<const float*>(p)));
    return f32x4{w.x, w.y, w.z, w.w};
  }

  // What was fetched of slice s to LDS at `to`.
  __device__ __forceinline__ void put(LIN_LDS char* to, const Held& h, int s, int wave, int lane) const {
    const bool k_ends = (s + 1) * BK > (KMAJOR ? rows : cols), hangs = KMAJOR && first + R > cols;
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      u32x4 lo = h.lo[t], hi;
      if (WIDE) hi = h.hi[t];
      if (k_ends || hangs) {  // uniform
        const int p = s * BK + place[t];
        const int by = KMAJOR ? down[t] : max(0, p + 8 - cols);
        if (by < 8) {
          move_down(lo, hi, by);
        } else {
          lo = 0;
          if (WIDE) hi = 0;
        }
        if (KMAJOR && p >= rows) {
          lo = 0;
          if (WIDE) hi = 0;
        }
      }
      if (WIDE) {
        const f32x4 a = __builtin_bit_cast(f32x4, lo), b = __builtin_bit_cast(f32x4, hi);
        lo = narrow8<TYPE>(f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
      }
      *(LIN_LDS u32x4*)(to + ((t * NW + wave) * 64 + lane) * 16) = lo;
    }
  }
  // Elements `by` .. 7 to 0 .., zeros behind them.
  static __device__ __forceinline__ void move_down(u32x4& lo, u32x4& hi, int by) {
    if constexpr (WIDE) {
      if (by & 4) lo = hi, hi = 0;
      if (by & 2) lo = u32x4{lo.z, lo.w, hi.x, hi.y}, hi = u32x4{hi.z, hi.w, 0, 0};
      if (by & 1) lo = u32x4{lo.y, lo.z, lo.w, hi.x}, hi = u32x4{hi.y, hi.z, hi.w, 0};
    } else {
      if (by & 4) lo = u32x4{lo.z, lo.w, 0, 0};
      if (by & 2) lo = u32x4{lo.y, lo.z, lo.w, 0};
      if (by & 1) lo = u32x4{lo.x >> 16 | lo.y << 16, lo.y >> 16 | lo.z << 16, lo.z >> 16 | lo.w << 16, lo.w >> 16};
    }
  }
};

template <int TYPE>
__device__ __forceinline__ float fragment_sum(s16x8 f) {
  const f32x8 v = widen8<TYPE>(__builtin_bit_cast(u32x4, f));
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// What a tile's sums become: eights of them at (row + d, col ..), from one place
// of a lane on.  What an eight needs from memory is fetched ahead of it.  ACT and
// BACKWARD are the launch's, RES whether it has a residual of y's 16-bit type (an
// fp32 one is read where it is added, registers being short).
template <int TYPE, int ACT, bool BACKWARD, bool RES>
struct LayerStore {
  static constexpr bool SLOPE = BACKWARD && ACT != LIN_ACT_NONE, FETCHES = SLOPE || RES;
  const LinEpilogue& e;
  const DropKey& key;
  const bool wide;  // y and the residual are fp32
  int64_t row, at_y, at_p, at_r;
  int col;
  f32x8 bias = 0.0f;
  struct Fetched {
    u32x4 z, r;
  };
  __device__ __forceinline__ LayerStore(const LinEpilogue& e_, const DropKey& k, int row_, int col_)
      : e(e_), key(k), wide(e_.y_type == GRAD_FP32), row(row_), col(col_) {
    at_y = row * e.ldy + col;
    at_p = row * e.ldp + col;
    at_r = row * e.ldr + col;
    if (!BACKWARD && e.bias) {
      bias = e.bias_type == GRAD_FP32 ? load8<GRAD_FP32>(e.bias, col) : load8<TYPE>(e.bias, col);
      asm volatile("" : "+v"(bias));  // waited for here, not after the stores of each part
    }
  }
  __device__ __forceinline__ Fetched fetch(int d) const {
    Fetched f;
    if constexpr (SLOPE) f.z = load_raw<TYPE>(e.preact, at_p + d * e.ldp);
    if constexpr (RES) f.r = load_raw<TYPE>(e.residual, at_r + d * e.ldr);
    return f;
  }
  // Until f is there.
  __device__ __forceinline__ void wait(Fetched& f) const {
    if constexpr (SLOPE) asm volatile("" : "+v"(f.z));
    if constexpr (RES) asm volatile("" : "+v"(f.r));
  }
  __device__ __forceinline__ void put(int d, f32x8 v, const Fetched& f) const {
    if constexpr (!BACKWARD) {
      v += bias;
      if (e.preact) store8<TYPE>(e.preact, at_p + d * e.ldp, v);
      v = act8<ACT>(v);
    } else if constexpr (SLOPE) {
      v = slope8<ACT>(widen8<TYPE>(f.z)) * v;
    }
    if (e.border != 0) v = drop8(e, key, row + d, col, v);
    if constexpr (RES) v = widen8<TYPE>(f.r) + v;
    if (!RES && wide) {
      if (e.residual) v = load8<GRAD_FP32>(e.residual, at_r + d * e.ldr) + v;
      store8<GRAD_FP32>(e.y, at_y + d * e.ldy, v);
    } else {
      store8<TYPE>(e.y, at_y + d * e.ldy, v);
    }
  }
};

// The same at the edges of the output: eights or single elements anywhere.
template <int TYPE>
struct LayerEdge {
  const LinEpilogue& e;
  const DropKey& key;
  __device__ __forceinline__ void eight(int64_t row, int col, f32x8 v) const {
    if (!e.backward) {
      if (e.bias) v += e.bias_type == GRAD_FP32 ? load8<GRAD_FP32>(e.bias, col) : load8<TYPE>(e.bias, col);
      if (e.preact) store8<TYPE>(e.preact, row * e.ldp + col, v);
      v = act8(v, e.act);
    } else if (e.act != LIN_ACT_NONE) {
      v = slope8(load8<TYPE>(e.preact, row * e.ldp + col), e.act) * v;
    }
    if (e.border != 0) v = drop8(e, key, row, col, v);
    if (e.y_type == GRAD_FP32) {
      if (e.residual) v = load8<GRAD_FP32>(e.residual, row * e.ldr + col) + v;
      store8<GRAD_FP32>(e.y, row * e.ldy + col, v);
    } else {
      if (e.residual) v = load8<TYPE>(e.residual, row * e.ldr + col) + v;
      store8<TYPE>(e.y, row * e.ldy + col, v);
    }
  }
  static __device__ __forceinline__ float get1(int type, const void* p, int64_t i) {
    return type == GRAD_FP32 ? load1<GRAD_FP32>(p, i) : load1<TYPE>(p, i);
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

template <bool ADD>
struct GradStore {
  static constexpr bool FETCHES = ADD;
  float* c;
  int64_t ldc, at;
  struct Fetched {
    f32x8 c;
  };
  __device__ __forceinline__ GradStore(float* c_, int64_t ldc_, int row, int col) : c(c_), ldc(ldc_), at(row * ldc_ + col) {}
  __device__ __forceinline__ Fetched fetch(int d) const {
    Fetched f;
    if constexpr (ADD) f.c = load8<GRAD_FP32>(c, at + d * ldc);
    return f;
  }
  __device__ __forceinline__ void wait(Fetched& f) const {
    if constexpr (ADD) asm volatile("" : "+v"(f.c));
  }
  __device__ __forceinline__ void put(int d, f32x8 v, const Fetched& f) const {
    if constexpr (ADD) v = f.c + v;
    store8<GRAD_FP32>(c, at + d * ldc, v);
  }
};

struct GradEdge {
  float* c;
  int64_t ldc;
  bool add;
  __device__ __forceinline__ void eight(int64_t row, int col, f32x8 v) const {
    if (add) v = load8<GRAD_FP32>(c, row * ldc + col) + v;
    store8<GRAD_FP32>(c, row * ldc + col, v);
  }
  __device__ __forceinline__ void one(int64_t row, int col, float v) const {
    if (add) v = load1<GRAD_FP32>(c, row * ldc + col) + v;
    store1<GRAD_FP32>(c, row * ldc + col, v);
  }
};

// How the operands reach LDS: by buffer loads; through registers; so, and B is fp32.
enum LinRead { READ_DIRECT = 0, READ_ANY = 1, READ_ANY_WIDE = 2 };

// BLOCKS: blocks a compute unit is to hold.
template <int TYPE, bool AK, bool BKM, bool GRAD, int BM, int BN, int BK, int WM, int WN, int WK, int NSTAGE, int BLOCKS, int READ = READ_DIRECT>
__global__ __launch_bounds__(64 * WM * WN * WK, WM * WN * WK * BLOCKS / 4) void linear_gemm_kernel(const LinGemmArgs a) {
  constexpr int NW = WM * WN * WK;
  constexpr int WTM = BM / WM, WTN = BN / WN;  // wave tile
  constexpr int TM = WTM / 16, TN = WTN / 16, PARTS = WTM / 32;
  typedef typename std::conditional<READ == READ_DIRECT, Slice<AK, BM, NW, BK>, AnySlice<TYPE, false, AK, BM, NW, BK>>::type SA;
  typedef typename std::conditional<READ == READ_DIRECT, Slice<BKM, BN, NW, BK>,
                                    AnySlice<TYPE, READ == READ_ANY_WIDE, BKM, BN, NW, BK>>::type SB;
  constexpr int STAGE = SA::BYTES + SB::BYTES;
  constexpr int PER = SA::LOADS + SB::LOADS;
  constexpr int STEPS = BK / 32 / WK;  // k-steps of a wave in a slice
  constexpr int PITCH = WTN * 4 + 16;  // staged fp32 rows: 16 bytes more move each row to other banks
  constexpr int AHEAD = PARTS > 1 && NW * 64 * PITCH <= 160 * 1024 / BLOCKS ? 2 : 1;  // 32-row parts of a wave tile staged at once
  constexpr int STAGED = NW * AHEAD * 32 * PITCH;
  constexpr int LDS = NSTAGE * STAGE > STAGED ? NSTAGE * STAGE : STAGED;
  static_assert(NSTAGE >= 2 && NSTAGE <= 8 && (NSTAGE - 1) * PER < 64 && LDS <= 160 * 1024, "ring");
  static_assert(STEPS >= 1 && STEPS * WK * 32 == BK && PARTS * 32 == WTM && TN * 16 == WTN, "wave tile");
  // Two sets of fragments, which change places within a slice, where registers
  // allow; two k-major operands and the sums of one leave too few of them for 256 x 256.
  constexpr bool READS_AHEAD = !(GRAD && TM * TN >= 32);
  static_assert(STEPS % 2 == 0 || STEPS == 1, "see READS_AHEAD");
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
  auto stage_of = [&](int s) { return (LIN_LDS char*)lds + (s % NSTAGE) * STAGE; };
  auto issue = [&](int s) {
    if constexpr (READ == READ_DIRECT) {
      const int have = a.k - (s0 + s) * BK;
      la.load(stage_of(s), have, wave, lane);
      lb.load(stage_of(s) + SA::BYTES, have, wave, lane);
    }
  };
  if constexpr (READ == READ_DIRECT) {
    la.start(a.a, row0, s0, wave, lane);
    lb.start(a.b, col0, s0, wave, lane);
#pragma unroll
    for (int s = 0; s < NSTAGE; ++s)
      if (s < slices) issue(s);
  } else {
    la.start(a.a, row0, a.m, a.k, wave, lane);
    lb.start(a.b, col0, a.n, a.k, wave, lane);
  }

  // The bias is read at the end of the tile: on its way to the L2 from here on.
  uint32_t touched = 0;
  if (!GRAD && a.e.bias) {
    const int col = min(col0 + wj * WTN + (lane * 8 & (WTN - 1)), a.n - 1);
    touched = *(gptr(static_cast<const uint16_t*>(a.e.bias)) + (a.e.bias_type == GRAD_FP32 ? 2 * (int64_t)col : col));
  }

  typename SA::Read ra[TM];
  typename SB::Read rb[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) ra[i] = SA::read_of(wi * WTM + i * 16, lane);
#pragma unroll
  for (int j = 0; j < TN; ++j) rb[j] = SB::read_of(wj * WTN + j * 16, lane);

  f32x4 acc[TM][TN];
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

  s16x8 fa[READS_AHEAD ? 2 : 1][TM], fb[READS_AHEAD ? 2 : 1][TN];
  auto read = [&](int s, int step, int set) {
    const LIN_LDS char* sa = stage_of(s);
    const int kk = WK == 1 ? step : step * WK + wk;
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[set][i] = SA::fragment(sa, ra[i], kk);
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[set][j] = SB::fragment(sa + SA::BYTES, rb[j], kk);
  };
  auto multiply = [&](int set) {
    // operands swapped: a lane then holds 4 consecutive columns of one row
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma<TYPE>(fb[set][j], fa[set][i], acc[i][j]);
  };

  auto add_sums = [&](int s) {
    if (!summing || (sharers != 1 && (s0 + s) % sharers != across)) return;
    const LIN_LDS char* sa = stage_of(s);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const int kk = WK == 1 ? t : t * WK + wk;
      if (a.sum_side == 1) {
#pragma unroll
        for (int j = 0; j < TN; ++j) sum[j] += fragment_sum<TYPE>(SB::fragment(sa + SA::BYTES, rb[j], kk));
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) sum[i] += fragment_sum<TYPE>(SA::fragment(sa, ra[i], kk));
      }
    }
  };

  // Slice s is there once this wave has only the loads of later slices
  // outstanding and every wave has passed a barrier.
  auto reduce = [&](auto works) {
    constexpr bool WORKS = decltype(works)::value;
    if (slices == 0) return;
    wait_slices<PER, NSTAGE + 1>(min(NSTAGE - 1, slices - 1));
    block_barrier();
    if constexpr (WORKS && READS_AHEAD) read(0, 0, 0);
#pragma unroll 1
    for (int s = 0; s < slices; ++s) {
      if constexpr (GRAD && WORKS) {
        add_sums(s);
      }
      if constexpr (WORKS && READS_AHEAD) {
#pragma unroll
        for (int t = 0; t < STEPS - 1; ++t) {
          read(s, t + 1, (t + 1) & 1);
          multiply(t & 1);
        }
      } else if constexpr (WORKS) {
#pragma unroll
        for (int t = 0; t < STEPS; ++t) {
          read(s, t, 0);
          if (t < STEPS - 1) multiply(0);
        }
      }
      if (s + 1 < slices) {
        // every wave has read all of slice s once it is here: its buffer is filled anew
        wait_slices<PER, NSTAGE>(min(NSTAGE - 2, slices - 2 - s));
        block_barrier();
        if (s + NSTAGE < slices) issue(s + NSTAGE);
        if constexpr (WORKS && READS_AHEAD && STEPS > 1) read(s + 1, 0, 0);
      }
      if constexpr (WORKS) {
        multiply(READS_AHEAD ? (STEPS - 1) & 1 : 0);
        if (READS_AHEAD && STEPS == 1 && s + 1 < slices) read(s + 1, 0, 0);
      }
    }
  };
  // Through registers: two LDS buffers, and two slices more on their way in registers.
  auto reduce_any = [&](auto works) {
    constexpr bool WORKS = decltype(works)::value;
    if constexpr (READ != READ_DIRECT) {
      static_assert(NSTAGE == 2, "one buffer is filled while the other is read");
      if (slices == 0) return;
      typename SA::Held ha[2];
      typename SB::Held hb[2];
      // behind the last slice, that one again: loads without a branch can be waited for one by one
      auto fetch = [&](int s, int set) __attribute__((always_inline)) {
        la.fetch(ha[set], s0 + min(s, slices - 1));
        lb.fetch(hb[set], s0 + min(s, slices - 1));
      };
      auto put = [&](int s, int set) __attribute__((always_inline)) {
        la.put(stage_of(set), ha[set], s0 + s, wave, lane);
        lb.put(stage_of(set) + SA::BYTES, hb[set], s0 + s, wave, lane);
      };
      auto step = [&](int s, int set) __attribute__((always_inline)) {
        // slice s is in LDS, and every wave has read all of the one before
        wait_loads<63>();
        block_barrier();
        if (s + 1 < slices) put(s + 1, set ^ 1);
        fetch(s + 3, set ^ 1);
        if constexpr (GRAD && WORKS) add_sums(s);
        if constexpr (WORKS) {
#pragma unroll
          for (int t = 0; t < STEPS; ++t) {
            read(s, t, 0);
            multiply(0);
          }
        }
      };
      fetch(0, 0);
      fetch(1, 1);
      put(0, 0);
      fetch(2, 0);
      for (int s = 0;; s += 2) {
        step(s, 0);
        if (s + 1 >= slices) break;
        step(s + 1, 1);
        if (s + 2 >= slices) break;
      }
    }
  };
  // A wave whose part of the tile lies outside the output only helps to load.
  const bool outside = row0 + wi * WTM >= a.m || col0 + wj * WTN >= a.n;
  if constexpr (READ != READ_DIRECT) {
    if (outside) reduce_any(std::false_type{});
    else reduce_any(std::true_type{});
  } else {
    if (outside) reduce(std::false_type{});
    else reduce(std::true_type{});
  }
  wait_loads<0>();
  if constexpr (!GRAD) asm volatile("" ::"v"(touched));
  block_barrier();

  // The sums go through LDS, 32 rows of each wave at a time, and are stored in
  // eights of consecutive columns, whole lines of the output: stored from
  // registers, 32 bytes to a row, a 16-bit output cost up to 1.4 times as much in all.
  constexpr int PART = 32 * PITCH, WAVE = AHEAD * PART, GROUP = WM * WN * WAVE;
  LIN_LDS char* staged = (LIN_LDS char*)lds + wave * WAVE;
  LIN_LDS char* first = (LIN_LDS char*)lds + (wave % (WM * WN)) * WAVE;  // of the wave tile's group wk = 0
  constexpr int EIGHTS = WTN / 8, AT_ONCE = 64 / EIGHTS;  // eights of a row, rows of the wave's lanes
  constexpr int MINE = 32 / (AT_ONCE * WK);               // eights of a lane in a part, AT_ONCE WK rows apart
  static_assert(AT_ONCE * EIGHTS == 64 && MINE * AT_ONCE * WK == 32, "each group of waves stores a share of the sums");
  static_assert((PARTS == AHEAD || PARTS == 2 * AHEAD) && (WK == 1 || PARTS == 1), "parts");
  const int row1 = row0 + wi * WTM + wk * AT_ONCE + lane / EIGHTS, col1 = col0 + wj * WTN + lane % EIGHTS * 8;
  const LIN_LDS char* mine = first + (wk * AT_ONCE + lane / EIGHTS) * PITCH + lane % EIGHTS * 32;
  // Parts from p on to LDS (p is a constant wherever this is used: registers take no index).
  auto stage = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          *(LIN_LDS f32x4*)(staged + q * PART + (16 * h + (lane & 15)) * PITCH + (j * 16 + 4 * (lane >> 4)) * 4) =
              acc[2 * (p + q) + h][j];
    if (WK > 1) {
      wait_loads<63>();
      block_barrier();
    }
  };
  // An eight, `d` rows below this lane's first, of the parts that are staged.
  auto staged_eight = [&](int d) __attribute__((always_inline)) {
    f32x8 x = 0.0f;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const LIN_LDS f32x4* p = (const LIN_LDS f32x4*)(mine + w * GROUP + d * PITCH);
      const f32x4 lo = p[0], hi = p[1];
      const f32x8 y = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      x = w == 0 ? y : x + y;
    }
    return x;
  };
  auto store_whole = [&](const auto& store) {
    typedef typename std::remove_cv<typename std::remove_reference<decltype(store)>::type>::type Store;
    typename Store::Fetched got[MINE], next[MINE];
    if constexpr (Store::FETCHES) {
#pragma unroll
      for (int t = 0; t < MINE; ++t) got[t] = store.fetch(t * AT_ONCE * WK);
    }
#pragma unroll
    for (int h = 0; h < PARTS; h += AHEAD) {
      stage(h);
#pragma clang loop unroll_count(GRAD ? AHEAD : 1)
      for (int i = h; i < h + AHEAD; ++i) {
        if constexpr (Store::FETCHES) {
          // what the next part needs goes out before this part's stores: waiting for
          // a load waits for all that went out before it
#pragma unroll
          for (int t = 0; t < MINE; ++t) {
            store.wait(got[t]);
            if (i + 1 < PARTS) next[t] = store.fetch(32 * (i + 1) + t * AT_ONCE * WK);
          }
        }
#pragma unroll
        for (int t = 0; t < MINE; ++t)
          store.put(32 * i + t * AT_ONCE * WK, staged_eight(32 * (i - h) + t * AT_ONCE * WK), got[t]);
        if constexpr (Store::FETCHES) {
#pragma unroll
          for (int t = 0; t < MINE; ++t) {
            store.wait(next[t]);
            got[t] = next[t];
          }
        }
      }
    }
  };
  auto store_edge = [&](const auto& edge) {
#pragma unroll
    for (int i = 0; i < PARTS; i += AHEAD) {
      stage(i);
#pragma unroll 1
      for (int u = 0; u < AHEAD * MINE; ++u) {
        const int d = u * AT_ONCE * WK, row = row1 + 32 * i + d;
        if (row < a.m && col1 + 8 <= a.n) edge.eight(row, col1, staged_eight(d));
      }
      const int c = a.n / 8 * 8 - col0 - wj * WTN, left = a.n % 8;  // the last columns, one by one
      if (left != 0 && c >= 0 && c < WTN) {
        for (int q = wk * 64 + lane; q < AHEAD * 32 * left; q += 64 * WK) {
          const int r = q / left, k = c + q - r * left, row = row0 + wi * WTM + 32 * i + r;
          if (row >= a.m) continue;
          const LIN_LDS char* at = first + r * PITCH + k * 4;
          float x = *(const LIN_LDS float*)at;
#pragma unroll
          for (int w = 1; w < WK; ++w) x += *(const LIN_LDS float*)(at + w * GROUP);
          edge.one(row, col0 + wj * WTN + k, x);
        }
      }
    }
  };
  const bool whole = row0 + BM <= a.m && col0 + BN <= a.n;
  if constexpr (!GRAD) {
    const DropKey key(a.e);
    if (a.splits > 1) {
      const int64_t ld = (int64_t)a.tiles_n * BN;
      float* part = a.part + split * (ld * a.tiles_m * BM);
      if (whole) store_whole(GradStore<false>(part, ld, row1, col1));
      else store_edge(GradEdge{part, ld, false});
    } else if (!whole) {
      store_edge(LayerEdge<TYPE>{a.e, key});
    } else {
      auto with_act = [&](auto backward, auto res) {
        constexpr bool BWD = decltype(backward)::value, RES = decltype(res)::value;
        switch (a.e.act) {
          case LIN_ACT_NONE: store_whole(LayerStore<TYPE, LIN_ACT_NONE, BWD, RES>(a.e, key, row1, col1)); break;
          case LIN_ACT_GELU: store_whole(LayerStore<TYPE, LIN_ACT_GELU, BWD, RES>(a.e, key, row1, col1)); break;
          case LIN_ACT_RELU: store_whole(LayerStore<TYPE, LIN_ACT_RELU, BWD, RES>(a.e, key, row1, col1)); break;
          default: store_whole(LayerStore<TYPE, LIN_ACT_RELU2, BWD, RES>(a.e, key, row1, col1));
        }
      };
      const bool res = a.e.residual && a.e.y_type != GRAD_FP32;
      if (a.e.backward) {
        if (res) with_act(std::true_type{}, std::true_type{});
        else with_act(std::true_type{}, std::false_type{});
      } else {
        if (res) with_act(std::false_type{}, std::true_type{});
        else with_act(std::false_type{}, std::false_type{});
      }
    }
  } else {
    const bool to_part = a.splits > 1;
    if (to_part) {  // rows padded to whole tiles
      const int64_t ld = (int64_t)a.tiles_n * BN;
      store_whole(GradStore<false>(a.part + split * (ld * a.tiles_m * BM), ld, row1, col1));
    } else if (whole) {
      if (a.add) store_whole(GradStore<true>(a.c, a.ldc, row1, col1));
      else store_whole(GradStore<false>(a.c, a.ldc, row1, col1));
    } else {
      store_edge(GradEdge{a.c, a.ldc, a.add != 0});
    }
    if (a.sum_side != 0) {
      const int edge = a.sum_side == 1 ? BN : BM, wt = a.sum_side == 1 ? WTN : WTM, frags = wt / 16;
      LIN_LDS float* red = (LIN_LDS float*)lds;  // WK x edge
      wait_loads<63>();
      block_barrier();
      if (summing) {
#pragma unroll
        for (int f = 0; f < TS; ++f) {
          if (f >= frags) break;
          float v = sum[f] + __shfl_xor(sum[f], 32);
          v += __shfl_xor(v, 16);
          if (lane < 16) red[wk * edge + (a.sum_side == 1 ? wj : wi) * wt + f * 16 + lane] = v;
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
