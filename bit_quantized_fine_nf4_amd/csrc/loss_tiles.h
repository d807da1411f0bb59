// Operand tiles of the head's products: copies from memory into LDS and MFMA fragments
// out of it (loss_gemm.hip, loss_wide.hip).
//
// The head W is the caller's row-major [V][h].  The compact hidden states and G live in the
// workspace and are blocked: 32 x 32 blocks of 2 KB, [token / 32][column / 32][32][32], rows
// past the last token zero up to the next 32.  A block is a contiguous stretch of whole
// cache lines whichever of its two indices is summed over.
//
// A tile enters a product in one of two ways:
//   rows   k runs along a row: a stage is [rows][BK] with 16-byte chunks XOR-swizzled by
//          row; a fragment (8 consecutive k of one row) is one 16-byte read;
//   cols   k runs down the rows: a fragment is two transposing reads (ds_read_b64_tr_b16),
//          whose 32-lane phases name 4 rows k of 64 bytes.  A stage of W is [BK][cols] as
//          it is, with 64-byte units XOR-swizzled by k % 4; a stage of blocks keeps them,
//          and 4 rows of a block are 256 consecutive bytes.  Either way a phase covers the
//          64 banks once.
// MFMA group kk of a stage takes k = 16 kk + 8 (lane / 32) + 0..7 of both operands.  Rows
// past an operand's end read as zero (buffer bounds).
// W's rows are copied 64 deep, in whole 128-byte lines.  (32-deep stages, half a line per
// copy, cost twice the cache requests: a copy-only loop moved 15 TB/s in half lines and 28
// TB/s in whole ones.)
#pragma once

#include "loss.h"

namespace ql {
namespace {

typedef short ls16x4 __attribute__((ext_vector_type(4)));

// Buffer descriptor over [base, base + bytes), for loads whose rows past the end read zero.
QL_DEV u32x4 lrsrc(const void *base, int64_t bytes) {
  const int64_t cap = 0x7FFFFFF0;
  const uint32_t n = (uint32_t)(bytes < 0 ? 0 : (bytes > cap ? cap : bytes));
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xFFFFu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)n), 0x00020000u};
}
QL_DEV f32x16 lmfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                0, 0);
}
// 16 bytes per lane from a buffer straight into LDS: lane L's bytes land at LDS address
// at + 16 L; at and soff are the wave's.  It has no register result, so nothing of the compiler's is in
// flight with it; its completion is awaited by the kernel's own vmcnt waits.  It is written
// in assembly because the compiler, which knows of the builtin that some LDS is being
// written, waits for every outstanding copy before each transposing LDS read: with it the
// dH and dW products of 4096 tokens x 8192 x 32000 took 2.4 and 2.2 instead of 1.6 ms.  (m0 is a reserved
// register that the compiler writes right before each use of its own; these kernels have
// none.)
// ONCE: nobody reads the bytes again (streamed past the caches' other contents).
template <bool ONCE = false>
QL_DEV void lload_lds(u32x4 rsrc, int at, int voff, int soff) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :
                 : "s"(at), "v"(voff), "s"(rsrc), "s"(soff));
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(at), "v"(voff), "s"(rsrc), "s"(soff));
}
QL_DEV u32x4 ltr_pair(const uint16_t *lo, const uint16_t *hi) {
  typedef __attribute__((address_space(3))) ls16x4 lds_s16x4;
  const ls16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lo));
  const ls16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(hi));
  const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
  return u32x4{ua[0], ua[1], ub[0], ub[1]};
}
// Workgroup barrier without the fences of __syncthreads(), which would wait for the
// copies in flight; the loop waits for what it needs itself.
QL_DEV void lbarrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr int kThreads = 256;
constexpr int kWaves = 4;

// An operand stored in rows: R rows of the tile, k along memory, BK of it per stage.
// A tile's descriptor (lrsrc) runs from its first row to the operand's end.  Row r's 16-byte
// chunks sit at chunk ^ f(r), so that the 16 lanes of a read phase (one chunk of 16
// consecutive rows) cover the 64 banks once.
template <int R, int BK, bool ONCE = false>
struct RowOperand {
  static constexpr int kElems = R * BK;
  static constexpr int CH = BK / 8;               // chunks per row
  static constexpr int kRows = 64 / CH;           // rows per 1 KB copy
  static constexpr int kBlocks = R / kRows;       // copies per stage
  static constexpr int kCopies = kBlocks < kWaves ? 1 : kBlocks / kWaves;  // per wave
  static_assert(kCopies == 1 || kCopies % 2 == 0, "a copy's swizzle depends on its parity");
  int voff[2], step;
  int frag, swz;
  static QL_DEV int f(int r) { return (r / (16 / CH)) & (CH - 1); }
  // with fewer copies than waves two waves make the same one: every wave's count of
  // outstanding copies stays the same
  static QL_DEV int block(int wv, int c) { return kBlocks < kWaves ? wv % kBlocks : wv * kCopies + c; }
  QL_DEV void init(int64_t ld, int lane, int wv, int first_row) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = kRows * block(wv, c) + lane / CH, lc = (lane % CH) ^ f(r);
      voff[c] = (int)((r * ld + lc * 8) * 2);
    }
    step = __builtin_amdgcn_readfirstlane((int)(kRows * ld * 2));
    const int r = first_row + (lane & 31);  // MFMA tiles are 32 rows apart: f is the same in all of them
    frag = r * BK;
    swz = f(r);
  }
  // copy c of stage kt into the slot at LDS address `at`
  QL_DEV void copy(const u32x4 &rsrc, int at, int wv, int kt_, int c) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_);
    lload_lds<ONCE>(rsrc, at + block(wv, c) * 1024, voff[c & 1], kt * BK * 2 + (c & ~1) * step);
  }
  QL_DEV u32x4 read(const uint16_t *stage, int lane, int t, int kk) const {
    return *reinterpret_cast<const u32x4 *>(stage + frag + t * 32 * BK + (((2 * kk + (lane >> 5)) ^ swz) << 3));
  }
};

// Blocked rows: R tokens of the tile, BK of the blocked columns per stage.  `ldb`: bytes
// of one row of blocks.
template <int R, int BK>
struct BlockRows {
  static constexpr int kElems = R * BK;
  static constexpr int CH = BK / 8, kRows = 64 / CH, kBlocks = R / kRows;
  static constexpr int kCopies = kBlocks < kWaves ? 1 : kBlocks / kWaves;
  int voff[2], ldb;
  int frag, swz;
  static QL_DEV int f(int r) { return RowOperand<R, BK>::f(r); }
  static QL_DEV int block(int wv, int c) { return RowOperand<R, BK>::block(wv, c); }
  QL_DEV void init(int64_t ld_bytes, int lane, int wv, int first_row) {
    ldb = __builtin_amdgcn_readfirstlane((int)ld_bytes);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = kRows * block(wv, c) + lane / CH, lc = (lane % CH) ^ f(r);
      voff[c] = (lc >> 2) * 2048 + (lane / CH) * 64 + (lc & 3) * 16;
    }
    const int r = first_row + (lane & 31);
    frag = r * BK;
    swz = f(r);
  }
  QL_DEV void copy(const u32x4 &rsrc, int at, int wv, int kt_, int c) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_), b = block(wv, c);
    lload_lds(rsrc, at + b * 1024, voff[c & 1],
              b / (32 / kRows) * ldb + b % (32 / kRows) * (kRows * 64) + kt * (BK / 32) * 2048);
  }
  QL_DEV u32x4 read(const uint16_t *stage, int lane, int t, int kk) const {
    return *reinterpret_cast<const u32x4 *>(stage + frag + t * 32 * BK + (((2 * kk + (lane >> 5)) ^ swz) << 3));
  }
};

// Blocked columns: C of the blocked columns along the tile, 32 tokens k per stage.
template <int C>
struct BlockCols {
  static constexpr int kElems = C * 32;
  static constexpr int kCopies = kElems / 512 / kWaves;
  int voff, ldb, frag;
  QL_DEV void init(int64_t ld_bytes, int lane, int, int first_col) {
    ldb = __builtin_amdgcn_readfirstlane((int)ld_bytes);
    voff = lane * 16;
    const int c = lane & 15, half = (lane >> 4) & 1, g = lane >> 5;
    frag = first_col * 32 + (8 * g + (c >> 2)) * 32 + 16 * half + 4 * (c & 3);
  }
  QL_DEV void copy(const u32x4 &rsrc, int at, int wv, int kt_, int c) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_);
    lload_lds(rsrc, at + (wv * kCopies + c) * 1024, voff, kt * ldb + (wv * kCopies + c) * 1024);
  }
  QL_DEV u32x4 read(const uint16_t *stage, int, int t, int kk) const {
    const uint16_t *lo = stage + frag + t * 1024 + kk * 512;
    return ltr_pair(lo, lo + 128);
  }
};

// An operand stored in columns: C columns of the tile along memory, k down the rows.  A
// row's 64-byte units sit at unit ^ (k % 4).
template <int C, int BK>
struct ColOperand {
  static constexpr int kElems = C * BK;
  static constexpr int kCopies = C * BK / 512 / kWaves;
  static constexpr int kPerCopy = 512 / C;        // rows k per 1 KB copy
  static constexpr int kLanes = 64 / kPerCopy;    // lanes (16-byte chunks) per row
  int voff[2], step, stride;
  int frag, unit;
  // (a descriptor's k rows are within 2^31 bytes: kernels walk longer sums in segments)
  QL_DEV void init(int64_t ld, int lane, int wv, int first_col) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = kPerCopy * (wv * kCopies + c) + lane / kLanes, pc = lane % kLanes;
      const int lc = (((pc >> 2) ^ (k & 3)) << 2) | (pc & 3);
      voff[c] = (int)((k * ld + lc * 8) * 2);
    }
    step = __builtin_amdgcn_readfirstlane((int)(kPerCopy * ld * 2));
    stride = __builtin_amdgcn_readfirstlane((int)(BK * ld * 2));
    const int c = lane & 15, half = (lane >> 4) & 1, g = lane >> 5;
    frag = (8 * g + (c >> 2)) * C + 16 * half + 4 * (c & 3);
    unit = (first_col >> 5) ^ (c >> 2);
  }
  QL_DEV void copy(const u32x4 &rsrc, int at, int wv, int kt_, int c) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_);
    lload_lds(rsrc, at + (wv * kCopies + c) * 1024, voff[c & 1], kt * stride + (c & ~1) * step);
  }
  // the first column's unit is a multiple of the wave's TA or TB (a power of two), so
  // unit + t is unit ^ t and the swizzle of tile t is the lane's with t XORed in
  QL_DEV u32x4 read(const uint16_t *stage, int, int t, int kk) const {
    const uint16_t *lo = stage + frag + 16 * kk * C + ((unit ^ t) << 5);
    return ltr_pair(lo, lo + 4 * C);
  }
};

// The longest stretch of k that a column operand with rows of ld values takes with 32-bit
// offsets, its copies past the end included.
QL_DEV int64_t col_segment(int64_t ld) {
  const int64_t k = (((int64_t)1 << 31) - 16) / (2 * ld) - 512;
  return k < 64 ? 64 : k / 64 * 64;
}

template <int TA, int TB>
QL_DEV void clear(f32x16 (&acc)[TA][TB]) {
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
}

// The element (row, col) of a blocked matrix with `blocks` blocks per row.
QL_DEV int64_t blocked(int64_t row, int64_t col, int64_t blocks) {
  return ((row >> 5) * blocks + (col >> 5)) * 1024 + (row & 31) * 32 + (col & 31);
}

// the row of accumulator element v in its 32 x 32 tile
QL_DEV int acc_row(int v, int g) { return 8 * (v >> 2) + 4 * g + (v & 3); }

}  // namespace
}  // namespace ql
