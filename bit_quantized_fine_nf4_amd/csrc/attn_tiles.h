// Tiles of keys, values, queries and output gradients in LDS, and the scores' steps that
// the attention kernels share (attn.hip, attn_bwd.hip, decode.hip).
//
// A tile is R rows (tokens) of one head, D values each (64 or 128; a narrower head's
// missing columns read as zero).  One copy in LDS serves both kinds of MFMA operand:
//   rows   8 consecutive values of one token: one 16-byte read;
//   cols   one value of 8 tokens: two transposing reads (ds_read_b64_tr_b16).
// A row's 16-byte chunks sit at chunk ^ fold(row).  The 16 lanes of a phase of a row read
// name one chunk of 16 consecutive rows, the 32 lanes of a transposing phase 4 rows of 64
// bytes (32-wide tiles) or 8 of 32 (16-wide ones): each covers the 64 banks once.
//
// A product that sums over tokens takes them in an order of its own.  The accumulator of a
// product whose rows are tokens holds, in lane half g, tokens 8 q + 4 g + e; those are
// elements 4 (q % 2) + e of the second product's operand in that lane, and the transposing
// reads fetch the other operand's tokens in the same order.  So weights go from one product
// to the next in registers, without a move between lanes.
#pragma once

#include "attn.h"
#include "loss_tiles.h"

#include <type_traits>

namespace ql {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// What is done to scores: nothing, a distance bias, or a cap and (its slope may be zero) a bias.
enum Form { kPlain, kBiased, kCapped };
inline Form form_of(float cap, const float *slopes) { return cap > 0.0f ? kCapped : slopes ? kBiased : kPlain; }

constexpr int kOutside = 0x7FFFFFF0;  // an offset past every descriptor's end

template <int D>
QL_DEV constexpr int fold(int r) {
  return D == 128 ? ((r & 3) << 2) | (((r >> 2) & 1) << 1) | ((r >> 3) & 1)
                  : (((r >> 1) & 1) << 2) | (((r >> 2) & 1) << 1) | ((r >> 3) & 1);
}

// Copies of a tile of 64 rows by four waves, or of 32 by two.  A lane's offset is its row's
// and its chunk's, whose swizzle the copy's number changes in two known bits.  HOLD: every
// copy's offset has a register; otherwise it is formed at each copy, where registers are
// what the sums lack.
template <int D, bool HOLD>
struct Tile {
  static constexpr int CH = D / 8;            // chunks per row
  static constexpr int kRows = 64 / CH;       // rows per 1 KB copy
  static constexpr int kCopies = 16 / kRows;  // per wave
  int row, chunk;                             // of copy 0, in bytes
  int off[HOLD ? kCopies : 1];
  QL_DEV int offset(int r, int k, int c, uint32_t width) const {
    const int e = k ^ (fold<D>(kRows * c) << 4);
    return e < (int)width ? r + e : kOutside;
  }
  QL_DEV void init(uint32_t pitch, uint32_t width, int lane, int wv) {
    const int r = kRows * wv * kCopies + lane / CH;
    row = r * (int)pitch;
    chunk = ((lane % CH) ^ fold<D>(r)) << 4;
    if constexpr (HOLD)
#pragma unroll
      for (int c = 0; c < kCopies; ++c) off[c] = offset(row, chunk, c, width);
  }
  // the tile into the slot at LDS address `at`
  QL_DEV void copy(const u32x4 &rsrc, int at, int wv, uint32_t pitch, uint32_t width) const {
    int r = row, k = chunk;
    if constexpr (!HOLD) asm volatile("" : "+v"(r), "+v"(k));  // (the compiler would form them before the loop)
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
      lload_lds<false, true>(rsrc, at + (wv * kCopies + c) * 1024, HOLD ? off[HOLD ? c : 0] : offset(r, k, c, width),
                kRows * c * (int)pitch);
  }
};
// A tensor's rows of one head, as the source of tiles.
struct TileSource {
  uint64_t base;
  uint32_t pitch, width;  // bytes between rows, of a row
  int rows;
  QL_DEV void init(const uint16_t *x, int64_t ld, int head, int d, int64_t M) {
    base = reinterpret_cast<uint64_t>(x + (int64_t)head * d);
    pitch = (uint32_t)(ld * 2);
    width = (uint32_t)d * 2;
    rows = (int)M;
  }
  // from row `first`: rows past the last read as zero (64 rows are within 2^28 bytes)
  QL_DEV u32x4 tile(int first) const {
    const uint64_t at = base + (uint64_t)(uint32_t)first * pitch;
    const int left = rows - first < 64 ? rows - first : 64;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xFFFFu)),
                 (uint32_t)__builtin_amdgcn_readfirstlane(left > 0 ? (int)((left - 1) * pitch + width) : 0),
                 0x00020000u};
  }
  template <int D, bool HOLD>
  QL_DEV void copy(const Tile<D, HOLD> &t, int first, int at, int wv) const {
    t.copy(tile(first), at, wv, pitch, width);
  }
};

// Reads of a tile.  A chunk's swizzle is an XOR of address bits above the lane's own part, so
// one base address a tile and the constants of the fragment give every address: held in
// registers they would not leave room for the sums.  Tiles begin at multiples of 1 KB.
typedef __attribute__((address_space(3))) const u32x4 LdsChunk;
typedef __attribute__((address_space(3))) ls16x4 LdsQuad;

template <int D>
struct Reader {
  uint32_t row, col;  // this lane's parts
  QL_DEV void init(int lane) {
    const int r = lane & 31, c = lane & 15, half = (lane >> 4) & 1, g = lane >> 5, q = 4 * g + (c >> 2);
    row = r * D * 2 + ((g ^ fold<D>(r & 15)) << 4);
    col = q * D * 2 + (((2 * half + ((c & 3) >> 1)) ^ fold<D>(q)) << 4) + 8 * (c & 1);
  }
};
// A 32 x 16 fragment: row 32 t + lane % 32, values 16 kk + 8 (lane / 32) + 0..7.
// `at`: the tile's address and the reader's row.
template <int D>
QL_DEV u32x4 row_frag(uint32_t at, int t, int kk) {
  return *(LdsChunk *)((at ^ (kk << 5)) + 32 * t * D * 2);
}
// Its transpose: value 32 t + lane % 32 of the 16 tokens from 16 b, in the accumulators' order.
template <int D>
QL_DEV u32x4 col_frag(uint32_t at, int t, int b) {
  const uint32_t lo = at ^ (t << 6), hi = at ^ (t << 6) ^ 16;  // (8 rows on, a chunk's swizzle differs in its lowest bit)
  const ls16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsQuad *)(lo + 16 * b * D * 2));
  const ls16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsQuad *)(hi + (16 * b + 8) * D * 2));
  const u32x2 ux = __builtin_bit_cast(u32x2, x), uy = __builtin_bit_cast(u32x2, y);
  return u32x4{ux[0], ux[1], uy[0], uy[1]};
}

// What is not finite in a tile, for a pass that has to tell what a query sees from what it does
// not.  A fragment with zeros in such places:
QL_DEV u32x4 finite(u32x4 x) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = (x[k] & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu;
    const uint32_t hi = (x[k] & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u;
    x[k] &= lo | hi;
  }
  return x;
}
// The rows of a tile (a bit each) that hold an infinity or a NaN:
template <int D, int R>
QL_DEV uint64_t odd_rows(uint32_t tile, int lane) {
  bool odd = false;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    const u32x4 x = *(LdsChunk *)(tile + lane % R * D * 2 + 16 * c);
#pragma unroll
    for (int k = 0; k < 4; ++k) odd = odd || (x[k] & 0x7F80u) == 0x7F80u || (x[k] & 0x7F800000u) == 0x7F800000u;
  }
  const uint64_t rows = __ballot(odd);
  return R == 64 ? rows : rows & ((1ull << (R & 63)) - 1);
}
// NaN into the sums of a lane that sees row r, where that row is not finite.
template <int D>
QL_DEV void spoil(f32x16 (&acc)[D / 32], uint32_t tile, int r, bool sees, int g) {
  typedef __attribute__((address_space(3))) const u32x2 LdsPair;
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x2 x = *(LdsPair *)(tile + r * D * 2 + (((4 * t + q) ^ fold<D>(r)) << 4) + 8 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = i & 1 ? bf16_hi(x[i >> 1]) : bf16_lo(x[i >> 1]);
        acc[t][4 * q + i] = __builtin_fmaf(sees ? v : 0.0f, 0.0f, acc[t][4 * q + i]);
      }
      __builtin_amdgcn_sched_barrier(0);  // (a few registers at a time)
    }
}

// Whether every value of the accumulators is finite.
template <int N>
QL_DEV bool all_finite(const f32x16 (&x)[N]) {
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) t = __builtin_fmaf(x[i][v], 0.0f, t);
  return t == 0.0f;
}
// Whether `mine` holds in any lane of the workgroup's `waves` waves (flags: one for each).
QL_DEV bool any_wave(bool mine, int *flags, int wave, int waves) {
  const bool here = __any(mine);
  if ((threadIdx.x & 63) == 0) flags[wave] = here;
  __syncthreads();
  bool all = false;
  for (int w = 0; w < waves; ++w) all = all || flags[w];
  return __builtin_amdgcn_readfirstlane(all);
}

// The fragments of 32 rows held in registers: row `row` (if it is one) of x, all values.
template <int D>
QL_DEV void load_rows(u32x4 (&f)[D / 16], const uint16_t *x, bool live, int d, int g) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const int e = 16 * kk + 8 * g;
    f[kk] = live && e < d ? *reinterpret_cast<const u32x4 *>(x + e) : u32x4{0, 0, 0, 0};
  }
}

// Values 8 v .. 8 v + 7 of an accumulator in bf16: the operand for 16 tokens.
QL_DEV u32x4 pack8(const f32x16 &x, int b) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[8 * b + 2 * i], x[8 * b + 2 * i + 1]);
  return o;
}

QL_DEV float both_halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
QL_DEV float both_halves_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                  false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// tanh(t) of x = 2 t log2(e), to a few roundings of itself however small it is: a capped score
// is the cap times it, so an error of the size of 1's rounding would grow with the cap.  From
// |t| = 1/2 on 1 - 2 / (exp(2 t) + 1), right at both ends (exp's 0 and infinity); below, where
// that cancels, x P(x^2) with P fitted to tanh(t) / x by least squares of the relative error at
// Chebyshev's points, which leaves 2^-26.  Scores of a cap in use hardly ever pass half of it, so
// a wave looks its values over first and takes the exponentials only if one does: step of 1531
// tokens, 24 heads of 64, cap 30 109 us, by exponentials alone 123, by both everywhere 141; of 2048
// tokens, 32 heads of 128, cap 30 253 (251), cap 4, which most tiles pass half of, 292 (257).
constexpr float kTanhSmall = 1.4426950408889634f;  // |x| at |t| = 1/2
template <bool FAR>
QL_DEV float tanh_of(float x) {
  const float s = x * x;
  float p = __builtin_fmaf(1.23535186e-06f, s, -3.18191771e-05f);
  p = __builtin_fmaf(p, s, 6.66246258e-04f);
  p = __builtin_fmaf(p, s, -1.38759156e-02f);
  p = x * __builtin_fmaf(p, s, 3.46573586e-01f);
  if constexpr (!FAR) return p;
  const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x) + 1.0f);
  return __builtin_fabsf(x) < kTanhSmall ? p : far;
}
// scores -> tanh of each times `in`
template <typename X, int N>
QL_DEV void tanh_all(X (&z)[N], float in) {
  constexpr int kEach = sizeof(X) / 4;
  float most = 0.0f;
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int v = 0; v < kEach; ++v) {
      z[t][v] *= in;
      most = fmaxf(most, __builtin_fabsf(z[t][v]));
    }
  if (__any(most >= kTanhSmall)) {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int v = 0; v < kEach; ++v) z[t][v] = tanh_of<true>(z[t][v]);
  } else {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int v = 0; v < kEach; ++v) z[t][v] = tanh_of<false>(z[t][v]);
  }
}

// Span of a query, clamped to the tokens; an empty one is (INT_MAX, 0), which sees nothing
// and leaves a union of spans as it is.
struct Span {
  int lo, hi;
};
QL_DEV Span span_of(const int32_t *spans, int64_t row, int64_t M) {
  Span s{0x7FFFFFFF, 0};
  if (row < M) {
    const int lo = spans[2 * row], hi = spans[2 * row + 1];
    const int l = lo < 0 ? 0 : lo, h = hi > (int)M ? (int)M : hi;
    if (l < h) s = Span{l, h};
  }
  return s;
}
// over the 32 rows that a wave holds in both halves: rotations within 16 lanes, then the
// other 16
QL_DEV int rows_min(int x) {
  auto turn = [](int v, auto by) { return __builtin_amdgcn_update_dpp(v, v, 0x120 + decltype(by)::value, 0xF, 0xF, false); };
  auto least = [](int a, int b) { return a < b ? a : b; };
  x = least(x, turn(x, std::integral_constant<int, 1>{}));
  x = least(x, turn(x, std::integral_constant<int, 2>{}));
  x = least(x, turn(x, std::integral_constant<int, 4>{}));
  x = least(x, turn(x, std::integral_constant<int, 8>{}));
  const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
  return __builtin_amdgcn_readfirstlane(least((int)r[0], (int)r[1]));
}
QL_DEV int rows_max(int x) { return -rows_min(-x); }

// The spans of a wave's 32 rows: keys that some row sees, and keys that every row sees that
// sees any (rows without a key have their results set apart).
struct Reach {
  int lo, hi;          // union
  int all_lo, all_hi;  // intersection
};
QL_DEV Reach reach_of(const Span &s) {
  const bool any = s.lo < s.hi;
  return Reach{rows_min(s.lo), rows_max(s.hi), rows_max(any ? s.lo : -0x7FFFFFFF), rows_min(any ? s.hi : 0x7FFFFFFF)};
}

// Workgroup -> (tile, head): with a multiple of eight heads each XCD (workgroups go to the
// eight in turn, each with its own L2) takes whole heads, so that the tiles of a head find
// its keys and values in L2 (so the steep heads of a geometric bias, whose dQ takes a pass more, are
// together on half of the XCDs).  Tiles are the slow index, so that the longest of all heads
// start first (2048 causal tokens, 64 heads, forward: 79 us; head after head 104).
QL_DEV void unit_place(int unit, int tiles, int heads, int &tile, int &head) {
  if ((heads & 7) == 0) {
    const int at = unit >> 3, each = heads >> 3;
    head = (unit & 7) * each + at % each;
    tile = at / each;
  } else {
    tile = unit / heads;
    head = unit % heads;
  }
}

// Eight consecutive values of one row from the two row groups 2 p and 2 p + 1 of an
// accumulator: lanes of the lower half get values 16 p .. + 7, of the upper half + 8 .. + 15.
QL_DEV u32x4 eight_of(const f32x16 &x, int p, float by) {
  const uint32_t a0 = pack_bf16x2(x[8 * p] * by, x[8 * p + 1] * by);
  const uint32_t a1 = pack_bf16x2(x[8 * p + 2] * by, x[8 * p + 3] * by);
  const uint32_t b0 = pack_bf16x2(x[8 * p + 4] * by, x[8 * p + 5] * by);
  const uint32_t b1 = pack_bf16x2(x[8 * p + 6] * by, x[8 * p + 7] * by);
  const auto u = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
  const auto v = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
  return u32x4{u[0], v[0], u[1], v[1]};
}
// Row `dst` of an output from accumulators whose columns are rows and rows are values;
// by 0: zeros, whatever the accumulators hold.
template <int D>
QL_DEV void store_row(uint16_t *dst, const f32x16 (&acc)[D / 32], float by, bool live, int d, int g) {
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      u32x4 v = eight_of(acc[t], p, by);
      if (by == 0.0f) v = u32x4{0, 0, 0, 0};
      const int e = 32 * t + 16 * p + 8 * g;
      if (live && e < d) *reinterpret_cast<u32x4 *>(dst + e) = v;
    }
}

// 4 bytes per lane from a buffer into LDS, as lload_lds.
QL_DEV void lload_lds4(u32x4 rsrc, int at, int voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(at), "v"(voff), "s"(rsrc));
}

// all of this wave's copies have landed and its LDS reads are done; then the workgroup's
QL_DEV void tile_sync() {
  __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0) lgkmcnt(0)
  lbarrier();
}

QL_DEV int lds_address(const void *p) {
  return __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)p);
}

template <int N>
QL_DEV void zero(f32x16 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) x[i][v] = 0.0f;
}

}  // namespace
}  // namespace ql
