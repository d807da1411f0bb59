// The products of the output head's cross entropy on 256 x 256 tiles, for gfx950:
//   logits  z = H · W^T   (a tile of z never leaves its workgroup: it becomes softmax
//                          statistics, or the gradient G in bf16)
//   dH      = G · W       (float32 partial sums over splits of the vocabulary)
//   dW      = G^T · H
// One persistent workgroup per compute unit: four waves, one per SIMD, 128 x 128 of the
// tile each (4 x 4 tiles of v_mfma_f32_32x32x16_bf16, 256 accumulator registers), both
// operands through LDS.  A workgroup walks its list of tiles as one stream of stages: the
// last stages of a tile copy the first of the next, so a tile costs neither a cold start
// nor copies past its end, and its epilogue runs while they land.
//
// LDS is all ring: ten slots of 256 x 32 (16 KB).  A blocked or column operand's stage is
// one slot; W's rows, copied 64 deep, take two (the logits: six slots for W, four for the
// hidden states; dH and dW five each).  A stage is two groups of 16 MFMAs, with one barrier
// between them: by then the stage's last fragments are read and its slots free.  The copies
// that follow are spread over the stage's second group and the next stage's first, one per
// four MFMAs: issued at once by all four waves they queue at the address unit and hold up
// the MFMAs behind them.  The barrier waits for the next stage only; two or three stages'
// copies stay in flight (2000 to 3000 cycles; a ring of three and two 64-deep stages left
// the second operand 1500, less than a miss takes: dW of 4096 x 8192 x 32000 1.81 ms).
//
// Bound by the matrix cores at the clock that their load leaves (about 1.8 GHz): busy 74, 75,
// 76 and 72 % of the cycles in the logits, the gradient, dH and dW of 4096 x 8192 x 32000,
// which take 1.65, 1.65, 1.65 and 1.72 ms (1.25 to 1.31 PFLOP/s); no LDS bank conflicts.
// With 1536 tokens 0.68, 0.68 and (dH, four splits) 0.72 ms; on a slower box 0.73, 0.73, 0.75.
//
// The MFMA's rows are the index that runs along the output's memory (the vocabulary for z
// and G, the hidden width for dH and dW): a lane then holds four consecutive outputs, and
// swapping halves between the two 32-lane groups makes 16-byte stores of eight.

#include "loss_tiles.h"

namespace ql {
namespace {

constexpr int kT = 256;              // tile edge
constexpr int kGroups = 256;         // workgroups: one per compute unit
constexpr int kSlot = kT * 32;       // elements of a slot
constexpr int kRingElems = 10 * kSlot;

// Item `i` of workgroup `wg`'s list -> unit number, -1 past the end.  Workgroups go to the
// eight XCDs in turn; each XCD takes a contiguous range of the units.
QL_DEV int unit_of(int wg, int i, int units) {
  const int per = (units + 7) / 8, l = (wg >> 3) + i * (kGroups / 8), u = (wg & 7) * per + l;
  return l < per && u < units ? u : -1;
}
// Tile (ta, tb) of place `u` in an order of bands of four tile rows, column by column: the
// 32 tiles that an XCD works on cover 4 x 8.
QL_DEV void tile_of(int u, int tiles_a, int tiles_b, int &ta, int &tb) {
  const int band = u / (4 * tiles_b);
  const int rows = tiles_a - 4 * band < 4 ? tiles_a - 4 * band : 4;
  const int r = u - 4 * band * tiles_b;
  tb = r / rows;
  ta = 4 * band + r % rows;
}

typedef f32x16 Acc[4][4];

// How an operand uses its part of the ring.  Stage s is 32 deep; a window is what follows
// stage s's barrier.  PAIR false: slot s % S, and the window copies stage s + S, four copies
// per wave.  PAIR true (64-deep copies): stages 2 P and 2 P + 1 share pair slot P % (S / 2),
// free after stage 2 P + 1; that window and the next copy the pair S / 2 further on, four of
// its eight copies each.
template <typename Op, int S, bool PAIR>
struct Lane {
  Op op;
  int at;               // element offset of its slots in the ring
  int slot;             // slot (pair: first of two) of the current double stage's first stage

  static QL_DEV int wrap(int s) { return s < S ? s : s - S; }
  static QL_DEV int back(int s) { return s >= 2 ? s - 2 : s + S - 2; }
  QL_DEV int elems(int s) const { return at + s * kSlot; }
  // fragment t of group kk (0..3) of the current double stage, or of the next (`ahead`)
  QL_DEV u32x4 read(const uint16_t *ring, int lane, int t, int kk, bool ahead) const {
    if (PAIR) return op.read(ring + elems(ahead ? wrap(slot + 2) : slot), lane, t, kk);
    return op.read(ring + elems(wrap(slot + (ahead ? 2 : 0) + (kk >> 1))), lane, t, kk & 1);
  }
  // copy c (0..3) of the window after stage `odd` (0, 1) of double stage d (`prev`: of the
  // double stage before the current one); rs and rn are this item's and the next one's
  // operand, nd this item's double stages
  QL_DEV void copy(int base, const u32x4 &rs, const u32x4 &rn, int nd, int d, int odd, bool prev, int wv, int c) const {
    const int cur = prev ? back(slot) : slot;
    if (PAIR) {
      // odd: the first half of pair d + S / 2 into this pair's slots; even: the second half
      // of pair d - 1 + S / 2 into the slots before
      const int P = (odd ? d : d - 1) + S / 2;
      op.copy(P < nd ? rs : rn, base + elems(odd ? cur : back(cur)) * 2, wv, P < nd ? P : P - nd, (odd ? 0 : 4) + c);
    } else {
      const int s = 2 * d + odd + S;
      op.copy(s < 2 * nd ? rs : rn, base + elems(wrap(cur + odd)) * 2, wv, s < 2 * nd ? s : s - 2 * nd, c);
    }
  }
  // the copies of the windows before the first stage, but for the last one's second half
  QL_DEV void fill(int base, const u32x4 &rs, int wv) {
    slot = 0;
    constexpr int units = PAIR ? S / 2 : S, each = PAIR ? 8 : 4;
#pragma unroll
    for (int s = 0; s < units; ++s)
#pragma unroll
      for (int c = 0; c < (s < units - 1 ? each : 2); ++c) op.copy(rs, base + elems(PAIR ? 2 * s : s) * 2, wv, s, c);
  }
};

// The stream of stages: ring, operands and the fragments of the next group.
template <typename LA, typename LB, int FLY>
struct Stream {
  LA A;
  LB B;
  uint16_t *ring;
  int base;  // its LDS address
  u32x4 fa[2][4], fb[2][4];

  QL_DEV void read(int kk, bool ahead, int f, int lane) {  // fragment f: A's, then B's
    if (f < 4) fa[kk & 1][f] = A.read(ring, lane, f, kk, ahead);
    else fb[kk & 1][f - 4] = B.read(ring, lane, f - 4, kk, ahead);
  }
  // this wave's copies of the next stage and its reads of this one are done; with that in
  // every wave, the next stage is whole and this one's slots are free
  static QL_DEV void sync() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((FLY & 15) | (7 << 4) | ((FLY >> 4) << 14));  // vmcnt(FLY) lgkmcnt(0)
    lbarrier();
    __builtin_amdgcn_sched_barrier(0);
  }

  QL_DEV void start(uint16_t *r, const u32x4 &ra, const u32x4 &rb, int lane, int wv) {
    ring = r;
    base = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)r);
    A.fill(base, ra, wv);
    B.fill(base, rb, wv);
    __builtin_amdgcn_s_waitcnt(0);
    lbarrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < 8; ++f) read(0, false, f, lane);
  }

  // One double stage (64 deep).
  QL_DEV void step(const u32x4 &ra, const u32x4 &na, const u32x4 &rb, const u32x4 &nb, int nd, int d, int lane, int wv,
                   Acc &acc) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        acc[m / 4][m % 4] = lmfma(fa[kk & 1][m / 4], fb[kk & 1][m % 4], acc[m / 4][m % 4]);
        // the next group's reads ride on this group's first half: done by its end
        if (m < 8) read((kk + 1) & 3, kk == 3, m, lane);
        // a window's first two copies of each operand follow the barrier (groups 1 and 3),
        // the other two ride on the next stage's first group (2 and 0)
        if (m % 4 == 3) {
          const int c = (kk & 1 ? 0 : 2) + (m >> 3), odd = kk == 1 || kk == 2 ? 0 : 1;
          const int dd = kk == 0 ? d - 1 : d;
          if (m & 4) B.copy(base, rb, nb, nd, dd, odd, kk == 0, wv, c);
          else A.copy(base, ra, na, nd, dd, odd, kk == 0, wv, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if ((kk & 1) == 0) sync();
    }
    A.slot = LA::wrap(A.slot + 2);
    B.slot = LB::wrap(B.slot + 2);
  }

  // An item of nd >= 3 double stages; na, nb: the next item's operands.
  QL_DEV void run(const u32x4 &ra, const u32x4 &rb, const u32x4 &na, const u32x4 &nb, int nd, int lane, int wv,
                  Acc &acc) {
    for (int d = 0; d < nd; ++d) step(ra, na, rb, nb, nd, d, lane, wv, acc);
  }
  QL_DEV void finish() {
    __builtin_amdgcn_s_waitcnt(0);  // no copy may land after the workgroup's end
  }
};

// Eight consecutive outputs of one column from the values of two row groups 2p and 2p + 1
// of an accumulator tile (a, b: this lane's four of each): lanes of the lower half get
// rows 16 p .. + 7, those of the upper half rows 16 p + 8 .. + 15.
QL_DEV u32x4 eight(const float (&a)[4], const float (&b)[4]) {
  const uint32_t a0 = pack_bf16x2(a[0], a[1]), a1 = pack_bf16x2(a[2], a[3]);
  const uint32_t b0 = pack_bf16x2(b[0], b[1]), b1 = pack_bf16x2(b[2], b[3]);
  const auto x = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
  return u32x4{x[0], y[0], x[1], y[1]};
}

// Stores in whole lines.  Lane l holds four pieces of row l % 32 of a wave's 32 x 32 (or 32 x
// 64) outputs; piece k of both 32-lane halves is 32 bytes of the row's 128.  Afterwards v[j]
// is row 8 row_group(j) + l % 8, and the piece is that of lane_piece(l): a store covers eight
// lines instead of a quarter of 32.  Lanes 16 apart are swapped first, then lanes 8 apart.
QL_DEV void by_lines(u32x4 (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; k += 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto x = __builtin_amdgcn_permlane16_swap(v[k][e], v[k + 1][e], false, false);
      v[k][e] = x[0];
      v[k + 1][e] = x[1];
    }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int a = (int)v[k][e], b = (int)v[k + 2][e];
      v[k][e] = (uint32_t)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xF, 0xC, false);  // row_ror:8
      v[k + 2][e] = (uint32_t)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xF, 0x3, false);
    }
}
QL_DEV constexpr int row_group(int j) { return (j >> 1) | (j & 1) << 1; }
QL_DEV int lane_piece(int lane) { return ((lane >> 4) & 1) | ((lane >> 3) & 1) << 1; }

}  // namespace

// GRAD false: part[half of a tile][token] = (max, sum of exp(z - max)) over 128
// vocabulary rows, and zlab of the tokens whose label is among them.
// GRAD true: G[token][v] = bf16((exp(z - lse) - [v is the label]) * (dloss / top)).
template <bool GRAD>
__global__ __launch_bounds__(kThreads) void head_logits_wide_kernel(LogitParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t ring[kRingElems];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count, tiles_t = (n + kT - 1) / kT, units = tiles_t * p.tiles_v;
  const int wg = blockIdx.x;
  int u = unit_of(wg, 0, units);
  if (u < 0) return;
  const int wa = (wv >> 1) * 128, wb = (wv & 1) * 128;
  // W's pairs of slots: three; the hidden states' slots: four.  At a barrier the copies of
  // two windows may be in flight.
  Stream<Lane<RowOperand<kT, 64>, 6, true>, Lane<BlockRows<kT, 32>, 4, false>, 16> S;
  S.A.op.init(p.h, lane, wv, wa);
  S.B.op.init(p.h * 64, lane, wv, wb);
  S.A.at = 0, S.B.at = 6 * kSlot;
  auto operands = [&](int unit, u32x4 &ra, u32x4 &rb) {
    int tv, tt;
    tile_of(unit, p.tiles_v, tiles_t, tv, tt);
    ra = lrsrc(p.W + (int64_t)tv * kT * p.h, (p.nvoc - (int64_t)tv * kT) * p.h * 2);
    rb = lrsrc(p.H + (int64_t)tt * kT * p.h, ((n + 31) / 32 * 32 - (int64_t)tt * kT) * p.h * 2);
  };
  u32x4 ra, rb, na, nb;
  operands(u, ra, rb);
  S.start(ring, ra, rb, lane, wv);
  const int nd = (int)(p.h / 64);
  const float top = GRAD ? *p.top : 0.0f;
  for (int i = 1; u >= 0; ++i) {
    const int next = unit_of(wg, i, units);
    operands(next >= 0 ? next : u, na, nb);
    Acc acc;
    clear(acc);
    S.run(ra, rb, na, nb, nd, lane, wv, acc);
    int tv, tt;
    tile_of(u, p.tiles_v, tiles_t, tv, tt);
    const int64_t v0 = (int64_t)tv * kT, t0 = (int64_t)tt * kT;
    // A lane holds rows 4 g + c of the wave's 128, c = 32 ii + 8 q + e known at compile time:
    // rows and labels are taken relative to 4 g, so that only c is compared with.
    const int lim = (int)(p.nvoc - v0 < kT ? p.nvoc - v0 : kT) - wa - 4 * g;  // rows of the vocabulary: c < lim
    const int vbase = (int)(p.v0 + v0) + wa + 4 * g;
    if constexpr (!GRAD) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + wb + 32 * j + l32;
        const int lab = t < n ? p.label[t] - vbase : -1;
        const bool mine = lab >= 0 && lab < 128 && !(lab & 4);  // (bit 2 set: the other half's)
        if (__any(mine)) {
          float z = 0.0f;
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int v = 0; v < 16; ++v) z = lab == 32 * ii + acc_row(v, 0) ? acc[ii][j][v] : z;
          if (mine) p.zlab[t] = z;
        }
        if (__any(lim < 128 - 4 * g)) {
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int v = 0; v < 16; ++v)
              if (32 * ii + acc_row(v, 0) >= lim) acc[ii][j][v] = -__builtin_inff();
        }
        float mx = -__builtin_inff();
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int v = 0; v < 16; ++v) mx = fmaxf(mx, acc[ii][j][v]);
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float ref = mx == -__builtin_inff() ? 0.0f : mx;  // no rows: the sum is 0
        float s = 0.0f;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int v = 0; v < 16; ++v) s += __expf(acc[ii][j][v] - ref);
        s += __shfl_xor(s, 32, 64);
        if (g == 0 && t < n) p.part[(2 * (int64_t)tv + (wv >> 1)) * p.ldp + t] = f32x2{mx, s};
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + wb + 32 * j + l32;
        const bool live = t < n;
        const float lse = live ? p.lse[t] : 0.0f;
        const float raw = live ? p.dloss[t] : 0.0f, dl = top > 0.0f ? raw / top : raw;
        const int lab = live ? p.label[t] - vbase : -1;
        // blocks of G: the wave's 32 tokens are one block row, tile ii one block (tokens past
        // the last: zero; the tile's rows are all there)
        uint16_t *dst = p.G + blocked(t, v0 + wa, p.gblocks) + 8 * g;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) {
            float o[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int c = 32 * ii + 16 * pp + 8 * q + e;
                const float pr = __expf(acc[ii][j][8 * pp + 4 * q + e] - lse);
                o[q][e] = c < lim ? (c == lab ? pr - 1.0f : pr) * dl : 0.0f;
              }
            *reinterpret_cast<u32x4 *>(dst + 1024 * ii + 16 * pp) = eight(o[0], o[1]);
          }
      }
    }
    u = next;
    ra = na, rb = nb;
  }
  S.finish();
}

// dH partial sums: part[split][token][c] (+)= sum over the split's vocabulary entries v of
// G[token][v] W[v][c].
__global__ __launch_bounds__(kThreads) void head_dh_wide_kernel(HeadGradParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t ring[kRingElems];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count, tiles_t = (n + kT - 1) / kT;
  const int tiles_h = (int)((p.h + kT - 1) / kT), tiles = tiles_t * tiles_h;
  const int splits = n > 0 ? head_splits(n, p.h, p.first, p.rows) : 0;
  const int units = tiles * splits, wg = blockIdx.x;
  const int nb64 = (int)((p.nvoc + 63) / 64);
  int u = unit_of(wg, 0, units);
  if (u < 0) return;
  const int wa = (wv >> 1) * 128, wb = (wv & 1) * 128;
  Stream<Lane<ColOperand<kT, 32>, 5, false>, Lane<BlockRows<kT, 32>, 5, false>, 24> S;
  S.A.op.init(p.h, lane, wv, wa);
  S.B.op.init(p.gblocks * 2048, lane, wv, wb);
  S.A.at = 0, S.B.at = 5 * kSlot;
  const int64_t seg = col_segment(p.h) / 64;  // blocks of 64 entries within 32-bit offsets
  // A unit's blocks [b0, b1) of 64 entries from block `from`: the operands and the number of
  // double stages.  W's rows from the range's end on read as zero, so three are always
  // right (G's columns there are written, or past its end).
  auto operands = [&](int unit, int64_t from, u32x4 &ra, u32x4 &rb, int &nd, int64_t &to) {
    int th, tt;
    tile_of(unit % tiles, tiles_h, tiles_t, th, tt);
    const int s = unit / tiles;
    const int64_t b0 = (int64_t)nb64 * s / splits, b1 = (int64_t)nb64 * (s + 1) / splits;
    const int64_t b = from < 0 ? b0 : from, e = b1 - b < seg ? b1 : b + seg;
    const int64_t k1 = e * 64 < p.nvoc ? e * 64 : p.nvoc;
    ra = lrsrc(p.W + b * 64 * p.h + (int64_t)th * kT, (k1 - b * 64) * p.h * 2 - (int64_t)th * kT * 2);
    const int64_t at = (int64_t)tt * (kT / 32) * p.gblocks + 2 * b;  // in blocks of 2 KB
    rb = lrsrc(p.G + at * 1024, ((n + 31) / 32 * p.gblocks - at) * 2048);
    nd = (int)(e - b > 3 ? e - b : 3);
    to = e < b1 ? e : -1;  // the unit goes on at block e
  };
  u32x4 ra, rb, na, nb;
  int nd, ndn;
  int64_t to, ton;
  operands(u, -1, ra, rb, nd, to);
  S.start(ring, ra, rb, lane, wv);
  for (int i = 1; u >= 0; ++i) {
    Acc acc;
    clear(acc);
    for (;;) {  // the unit's segments
      const int next = to >= 0 ? u : unit_of(wg, i, units);
      operands(next >= 0 ? next : u, to, na, nb, ndn, ton);
      S.run(ra, rb, na, nb, nd, lane, wv, acc);
      const bool more = to >= 0;
      ra = na, rb = nb, nd = ndn, to = ton;
      if (!more) break;
    }
    {
      int th, tt;
      tile_of(u % tiles, tiles_h, tiles_t, th, tt);
      float *out = p.part + (int64_t)(u / tiles) * n * p.h;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t0 = (int64_t)tt * kT + wb + 32 * j + (lane & 7);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          u32x4 w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = __builtin_bit_cast(u32x4, f32x4{acc[ii][j][4 * q], acc[ii][j][4 * q + 1], acc[ii][j][4 * q + 2],
                                                   acc[ii][j][4 * q + 3]});
          by_lines(w);
          const int64_t c = (int64_t)th * kT + wa + 32 * ii + 8 * lane_piece(lane) + 4 * g;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t t = t0 + 8 * row_group(k);
            if (t >= n || c >= p.h) continue;
            f32x4 v = __builtin_bit_cast(f32x4, w[k]);
            float *dst = out + t * p.h + c;
            if (p.add) v += *reinterpret_cast<const f32x4 *>(dst);
            *reinterpret_cast<f32x4 *>(dst) = v;
          }
        }
      }
    }
    u = unit_of(wg, i, units);
  }
  S.finish();
}

// dW[v][c] = bf16(top * sum over the tokens of G[token][v] H[token][c]).
__global__ __launch_bounds__(kThreads) void head_dw_wide_kernel(HeadGradParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t ring[kRingElems];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  const int tiles_h = (int)((p.h + kT - 1) / kT), tiles_v = (int)((p.nvoc + kT - 1) / kT);
  const int units = tiles_h * tiles_v, wg = blockIdx.x;
  int u = unit_of(wg, 0, units);
  if (u < 0) return;
  const int wa = (wv >> 1) * 128, wb = (wv & 1) * 128;
  Stream<Lane<BlockCols<kT>, 5, false>, Lane<BlockCols<kT>, 5, false>, 24> S;
  S.A.op.init(p.h * 64, lane, wv, wa);
  S.B.op.init(p.gblocks * 2048, lane, wv, wb);
  S.A.at = 0, S.B.at = 5 * kSlot;
  const int blocks = (n + 63) / 64, rows32 = (n + 31) / 32;
  // 64-token steps within 32-bit offsets, the copies past the end included
  const int64_t wide = p.h * 64 > p.gblocks * 2048 ? p.h * 64 : p.gblocks * 2048;
  const int64_t seg = (((int64_t)1 << 31) - 65536) / (2 * wide) - 4;
  // both operands are zero from token n to the next 32 and read as zero from there on
  auto operands = [&](int unit, int64_t from, u32x4 &ra, u32x4 &rb, int &nd, int64_t &to) {
    int th, tv;
    tile_of(unit, tiles_h, tiles_v, th, tv);
    const int64_t b = from < 0 ? 0 : from, e = blocks - b < seg ? blocks : b + seg;
    const int64_t ha = 2 * b * (p.h / 32) + th * (kT / 32), ga = 2 * b * p.gblocks + tv * (kT / 32);  // in blocks
    ra = lrsrc(p.H + ha * 1024, (rows32 * (p.h / 32) - ha) * 2048);
    rb = lrsrc(p.G + ga * 1024, (rows32 * p.gblocks - ga) * 2048);
    nd = (int)(e - b > 3 ? e - b : 3);
    to = e < blocks ? e : -1;
  };
  u32x4 ra, rb, na, nb;
  int nd, ndn;
  int64_t to, ton;
  operands(u, -1, ra, rb, nd, to);
  S.start(ring, ra, rb, lane, wv);
  const float top = n > 0 ? *p.top : 0.0f;
  for (int i = 1; u >= 0; ++i) {
    Acc acc;
    clear(acc);
    for (;;) {  // the unit's segments
      const int next = to >= 0 ? u : unit_of(wg, i, units);
      operands(next >= 0 ? next : u, to, na, nb, ndn, ton);
      S.run(ra, rb, na, nb, nd, lane, wv, acc);
      const bool more = to >= 0;
      ra = na, rb = nb, nd = ndn, to = ton;
      if (!more) break;
    }
    {
      int th, tv;
      tile_of(u, tiles_h, tiles_v, th, tv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t v0 = (int64_t)tv * kT + wb + 32 * j + (lane & 7);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          u32x4 w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float o[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[q][e] = top * acc[2 * half + (k >> 1)][j][8 * (k & 1) + 4 * q + e];
            w[k] = eight(o[0], o[1]);
          }
          by_lines(w);
          const int64_t c = (int64_t)th * kT + wa + 64 * half + 16 * lane_piece(lane) + 8 * g;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t v = v0 + 8 * row_group(k);
            if (v < p.nvoc && c < p.h) *reinterpret_cast<u32x4 *>(p.dW + v * p.h + c) = w[k];
          }
        }
      }
    }
    u = unit_of(wg, i, units);
  }
  S.finish();
}

hipError_t launch_logit_wide(LogitParams &p, bool grad, hipStream_t st) {
  p.tiles_v = (int)((p.nvoc + kT - 1) / kT);
  return grad ? launch(head_logits_wide_kernel<true>, kGroups, kThreads, st, p)
              : launch(head_logits_wide_kernel<false>, kGroups, kThreads, st, p);
}

hipError_t launch_head_dh_wide(HeadGradParams &p, hipStream_t st) {
  return launch(head_dh_wide_kernel, kGroups, kThreads, st, p);
}

hipError_t launch_head_dw(HeadGradParams &p, hipStream_t st) {
  return launch(head_dw_wide_kernel, kGroups, kThreads, st, p);
}

}  // namespace ql
