// The products of the output head's cross entropy on 256 x 256 tiles, for gfx950:
//   logits  z = H · W^T   (a tile of z never leaves its workgroup: it becomes softmax
//                          statistics, or the gradient G in bf16)
//   dH      = G · W       (float32 partial sums over splits of the vocabulary)
//   dW      = G^T · H
// One persistent workgroup per compute unit: four waves, one per SIMD, 128 x 128 of the
// tile each (4 x 4 tiles of v_mfma_f32_32x32x16_bf16, 256 accumulator registers), both
// operands through LDS.  A workgroup walks its list of tiles as one stream of 64-deep
// stages: the last two stages of a tile copy the first two of the next, so a tile costs
// neither a cold start nor copies past its end, and its epilogue runs while they land.
//
// LDS is all ring: three slots for operand A and two for B (160 KB).  Stage kt's slots are
// free after its barrier, which follows its third group of MFMAs: by then its last
// fragments are read.  B's copy of stage kt + 2 is issued in the last group, A's in the
// next stage's groups, so that copies are spread over the stage: issued at once by all
// four waves they queue at the address unit and hold up the MFMAs behind them.  The
// barrier waits for the copies of stage kt + 1 and lets A's of stage kt + 2 fly.
//
// The MFMA's rows are the index that runs along the output's memory (the vocabulary for z
// and G, the hidden width for dH and dW): a lane then holds four consecutive outputs, and
// swapping halves between the two 32-lane groups makes 16-byte stores of eight.

#include "loss_tiles.h"

namespace ql {
namespace {

constexpr int kT = 256;             // tile edge
constexpr int kWideBK = 64;
constexpr int kGroups = 256;        // workgroups: one per compute unit
constexpr int kSlotsA = 3, kSlotsB = 2;
constexpr int kRingElems = (kSlotsA + kSlotsB) * kT * kWideBK;

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

// The stream of stages: ring position and the fragments of the next group.
template <typename OpA, typename OpB>
struct Stream {
  OpA A;
  OpB B;
  uint16_t *ring;
  int base;     // its LDS address
  int sa, sb;   // slots of the current stage
  u32x4 fa[2][4], fb[2][4];

  QL_DEV void read(int slot_a, int slot_b, int kk, int set, int f, int lane) {  // fragment f: A's, then B's
    if (f < 4) fa[set][f] = A.read(ring + slot_a * OpA::kElems, lane, f, kk);
    else fb[set][f - 4] = B.read(ring + kSlotsA * OpA::kElems + slot_b * OpB::kElems, lane, f - 4, kk);
  }
  QL_DEV void copy_a(const u32x4 &rs, int slot, int wv, int kt, int c) const {
    A.copy(rs, base + slot * OpA::kElems * 2, wv, kt, c);
  }
  QL_DEV void copy_b(const u32x4 &rs, int slot, int wv, int kt, int c) const {
    B.copy(rs, base + (kSlotsA * OpA::kElems + slot * OpB::kElems) * 2, wv, kt, c);
  }
  static QL_DEV int up(int s, int n, int slots) { return s + n < slots ? s + n : s + n - slots; }

  // this wave's copies of the next stage and its reads of this one are done; with that in
  // every wave, the next stage is whole and this one's slots are free
  static QL_DEV void sync() {
    constexpr int kFly = OpA::kCopies;  // A's copies of the stage after the next
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((kFly & 15) | (7 << 4) | ((kFly >> 4) << 14));  // and lgkmcnt(0)
    lbarrier();
    __builtin_amdgcn_sched_barrier(0);
  }

  // the first item's stages 0 and 1, in the order in which the loop issues later ones
  QL_DEV void start(const u32x4 &ra, const u32x4 &rb, int lane, int wv) {
    sa = sb = 0;
#pragma unroll
    for (int c = 0; c < OpA::kCopies; ++c) copy_a(ra, 0, wv, 0, c);
#pragma unroll
    for (int c = 0; c < OpB::kCopies; ++c) copy_b(rb, 0, wv, 0, c);
#pragma unroll
    for (int c = 0; c < OpA::kCopies; ++c) copy_a(ra, 1, wv, 1, c);
#pragma unroll
    for (int c = 0; c < OpB::kCopies; ++c) copy_b(rb, 1, wv, 1, c);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(((OpA::kCopies + OpB::kCopies) & 15) | (7 << 4) | (15 << 8) |
                               (((OpA::kCopies + OpB::kCopies) >> 4) << 14));
    lbarrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < 8; ++f) read(0, 0, 0, 0, f, lane);
  }

  // One stage: multiplies it and copies stage `kc` of the item behind ra, rb (two stages
  // further along the stream).
  QL_DEV void step(const u32x4 &ra, const u32x4 &rb, int kc, int lane, int wv, Acc &acc) {
    const int sa1 = up(sa, 1, kSlotsA), sa2 = up(sa, 2, kSlotsA), sb1 = sb ^ 1;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const bool last = kk == 3;
      const int c0 = last ? 0 : OpA::kCopies * kk / 3, c1 = last ? OpB::kCopies : OpA::kCopies * (kk + 1) / 3;
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        acc[m / 4][m % 4] = lmfma(fa[kk & 1][m / 4], fb[kk & 1][m % 4], acc[m / 4][m % 4]);
        // the next group's reads ride on this group's first half: done by its end
        if (m < 8) read(last ? sa1 : sa, last ? sb1 : sb, last ? 0 : kk + 1, (kk + 1) & 1, m, lane);
#pragma unroll
        for (int c = c0 + (c1 - c0) * m / 16; c < c0 + (c1 - c0) * (m + 1) / 16; ++c) {
          if (last) copy_b(rb, sb, wv, kc, c);
          else copy_a(ra, sa2, wv, kc, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kk == 2) sync();
    }
    sa = sa1;
    sb = sb1;
  }

  // An item of nk >= 2 stages; `na`, `nb` are the next item's operands.
  QL_DEV void run(const u32x4 &ra, const u32x4 &rb, const u32x4 &na, const u32x4 &nb, int nk, int lane, int wv,
                  Acc &acc) {
    for (int kt = 0; kt < nk - 2; ++kt) step(ra, rb, kt + 2, lane, wv, acc);
    step(na, nb, 0, lane, wv, acc);
    step(na, nb, 1, lane, wv, acc);
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

}  // namespace

// GRAD false: part[64 K-row half of a tile][token] = (max, sum of exp(z - max)) over 128
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
  Stream<RowOperand<kT, kWideBK>, RowOperand<kT, kWideBK>> S;
  S.ring = ring;
  S.base = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)ring);
  S.A.init(p.h, lane, wv, wa);
  S.B.init(p.h, lane, wv, wb);
  auto operands = [&](int unit, u32x4 &ra, u32x4 &rb) {
    int tv, tt;
    tile_of(unit, p.tiles_v, tiles_t, tv, tt);
    ra = lrsrc(p.W + (int64_t)tv * kT * p.h, (p.nvoc - (int64_t)tv * kT) * p.h * 2);
    rb = lrsrc(p.H + (int64_t)tt * kT * p.h, ((int64_t)n - (int64_t)tt * kT) * p.h * 2);
  };
  u32x4 ra, rb, na, nb;
  operands(u, ra, rb);
  S.start(ra, rb, lane, wv);
  const int nk = (int)(p.h / kWideBK);
  const float top = GRAD ? *p.top : 0.0f;
  for (int i = 1; u >= 0; ++i) {
    const int next = unit_of(wg, i, units);
    operands(next >= 0 ? next : u, na, nb);
    Acc acc;
    clear(acc);
    S.run(ra, rb, na, nb, nk, lane, wv, acc);
    int tv, tt;
    tile_of(u, p.tiles_v, tiles_t, tv, tt);
    const int64_t v0 = (int64_t)tv * kT, t0 = (int64_t)tt * kT;
    const int rows = (int)(p.nvoc - v0 < kT ? p.nvoc - v0 : kT) - wa;  // vocabulary rows of this wave's 128
    if constexpr (!GRAD) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + wb + 32 * j + l32;
        // the label's place among this wave's rows (outside [0, 128): not here)
        const int64_t lab = t < n ? (int64_t)p.label[t] - p.v0 - v0 - wa : -1;
        if (__any(lab >= 0 && lab < 128)) {
          float z = 0.0f;
          const int l = (int)lab - 4 * g;  // rows 32 i + 8 q + e of the lane's half
          bool mine = false;
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const bool hit = l == 32 * ii + acc_row(v, 0) && lab >= 0 && lab < 128;
              z = hit ? acc[ii][j][v] : z;
              mine |= hit;
            }
          if (mine) p.zlab[t] = z;
        }
        if (rows < 128) {
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int v = 0; v < 16; ++v)
              if (32 * ii + acc_row(v, g) >= rows) acc[ii][j][v] = -__builtin_inff();
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
        const float lse = live ? p.lse[t] : 0.0f, dl = live && top > 0.0f ? p.dloss[t] / top : 0.0f;
        const int64_t lab = live ? (int64_t)p.label[t] - p.v0 - v0 - wa : -1;
        uint16_t *dst = p.G + t * p.ldg + v0 + wa + 8 * g;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) {
            float o[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int row = 32 * ii + 16 * pp + 8 * q + 4 * g + e;
                const float pr = __expf(acc[ii][j][8 * pp + 4 * q + e] - lse);
                o[q][e] = row < rows ? (row == lab ? pr - 1.0f : pr) * dl : 0.0f;
              }
            const u32x4 w = eight(o[0], o[1]);  // every lane: the swap needs both halves
            if (live) *reinterpret_cast<u32x4 *>(dst + 32 * ii + 16 * pp) = w;
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
  Stream<ColOperand<kT, kWideBK>, RowOperand<kT, kWideBK>> S;
  S.ring = ring;
  S.base = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)ring);
  S.A.init(p.h, lane, wv, wa);
  S.B.init(p.ldg, lane, wv, wb);
  const int64_t seg = col_segment(p.h) / 64;  // blocks of 64 entries within 32-bit offsets
  // A unit's blocks [b0, b1) from block `from`: the operands and the number of stages.  W's
  // rows from the range's end on read as zero, so two stages are always right.
  auto operands = [&](int unit, int64_t from, u32x4 &ra, u32x4 &rb, int &nk, int64_t &to) {
    int th, tt;
    tile_of(unit % tiles, tiles_h, tiles_t, th, tt);
    const int s = unit / tiles;
    const int64_t b0 = (int64_t)nb64 * s / splits, b1 = (int64_t)nb64 * (s + 1) / splits;
    const int64_t b = from < 0 ? b0 : from, e = b1 - b < seg ? b1 : b + seg;
    const int64_t k1 = e * 64 < p.nvoc ? e * 64 : p.nvoc;
    ra = lrsrc(p.W + b * 64 * p.h + (int64_t)th * kT, (k1 - b * 64) * p.h * 2 - (int64_t)th * kT * 2);
    rb = lrsrc(p.G + (int64_t)tt * kT * p.ldg + b * 64, ((int64_t)n - (int64_t)tt * kT) * p.ldg * 2 - b * 128);
    nk = (int)(e - b > 2 ? e - b : 2);
    to = e < b1 ? e : -1;  // the unit goes on at block e
  };
  u32x4 ra, rb, na, nb;
  int nk, nkn;
  int64_t to, ton;
  operands(u, -1, ra, rb, nk, to);
  S.start(ra, rb, lane, wv);
  Acc acc;
  clear(acc);
  for (int i = 1; u >= 0;) {
    const int next = to >= 0 ? u : unit_of(wg, i, units);
    operands(next >= 0 ? next : u, to, na, nb, nkn, ton);
    S.run(ra, rb, na, nb, nk, lane, wv, acc);
    if (to < 0) {
      int th, tt;
      tile_of(u % tiles, tiles_h, tiles_t, th, tt);
      float *out = p.part + (int64_t)(u / tiles) * n * p.h;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = (int64_t)tt * kT + wb + 32 * j + l32;
        float *dst = out + t * p.h;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int64_t c = (int64_t)th * kT + wa + 32 * ii + 8 * q + 4 * g;
            if (t >= n || c >= p.h) continue;
            f32x4 v{acc[ii][j][4 * q], acc[ii][j][4 * q + 1], acc[ii][j][4 * q + 2], acc[ii][j][4 * q + 3]};
            if (p.add) v += *reinterpret_cast<const f32x4 *>(dst + c);
            *reinterpret_cast<f32x4 *>(dst + c) = v;
          }
      }
      clear(acc);
      ++i;
    }
    u = next;
    ra = na, rb = nb, nk = nkn, to = ton;
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
  Stream<ColOperand<kT, kWideBK>, ColOperand<kT, kWideBK>> S;
  S.ring = ring;
  S.base = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)ring);
  S.A.init(p.h, lane, wv, wa);
  S.B.init(p.ldg, lane, wv, wb);
  const int blocks = (n + 63) / 64;
  const int64_t seg = col_segment(p.h > p.ldg ? p.h : p.ldg) / 64;
  // both operands read as zero from token n on
  auto operands = [&](int unit, int64_t from, u32x4 &ra, u32x4 &rb, int &nk, int64_t &to) {
    int th, tv;
    tile_of(unit, tiles_h, tiles_v, th, tv);
    const int64_t b = from < 0 ? 0 : from, e = blocks - b < seg ? blocks : b + seg, t = b * 64;
    ra = lrsrc(p.H + t * p.h + (int64_t)th * kT, (n - t) * p.h * 2 - (int64_t)th * kT * 2);
    rb = lrsrc(p.G + t * p.ldg + (int64_t)tv * kT, (n - t) * p.ldg * 2 - (int64_t)tv * kT * 2);
    nk = (int)(e - b > 2 ? e - b : 2);
    to = e < blocks ? e : -1;
  };
  u32x4 ra, rb, na, nb;
  int nk, nkn;
  int64_t to, ton;
  operands(u, -1, ra, rb, nk, to);
  S.start(ra, rb, lane, wv);
  const float top = n > 0 ? *p.top : 0.0f;
  Acc acc;
  clear(acc);
  for (int i = 1; u >= 0;) {
    const int next = to >= 0 ? u : unit_of(wg, i, units);
    operands(next >= 0 ? next : u, to, na, nb, nkn, ton);
    S.run(ra, rb, na, nb, nk, lane, wv, acc);
    if (to < 0) {
      int th, tv;
      tile_of(u, tiles_h, tiles_v, th, tv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t v = (int64_t)tv * kT + wb + 32 * j + l32;
        uint16_t *dst = p.dW + v * p.h;
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) {
            float o[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[q][e] = top * acc[ii][j][8 * pp + 4 * q + e];
            const u32x4 w = eight(o[0], o[1]);
            const int64_t c = (int64_t)th * kT + wa + 32 * ii + 16 * pp + 8 * g;
            if (v < p.nvoc && c < p.h) *reinterpret_cast<u32x4 *>(dst + c) = w;
          }
      }
      clear(acc);
      ++i;
    }
    u = next;
    ra = na, rb = nb, nk = nkn, to = ton;
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
