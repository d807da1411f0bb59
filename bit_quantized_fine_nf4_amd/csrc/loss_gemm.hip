// The matrix products behind the cross entropy of an output head, for gfx950:
//   logits  z = H · W^T           (tile of z never leaves the workgroup: it becomes
//                                  softmax statistics, or the gradient G in bf16)
//   dH      = G · W               (split over the vocabulary, float32 partial sums)
//   dW      = G^T · H
// One main loop serves all three.  Four waves (one per SIMD) share a tile through LDS;
// each computes TA x TB MFMA tiles of 32 x 32 (v_mfma_f32_32x32x16_bf16), BK deep per
// stage.  Both operands go from memory straight into LDS (buffer_load ... lds, 16 bytes
// per lane) in a ring of stages.  An operand is stored in one of two ways:
//   rows   k runs along memory: a stage is [rows][BK] with 16-byte chunks XOR-swizzled
//          by row; a fragment (8 consecutive k of one row) is
//          one 16-byte read;
//   cols   the tile's own index runs along memory: a stage is [BK][cols] as it is,
//          whose 64-byte units are XOR-swizzled by k % 4; a fragment is two transposing
//          reads (ds_read_b64_tr_b16), whose 32-lane phases name 4 rows k of one unit
//          and so cover the 64 banks once.
// MFMA group kk of a stage takes k = 16 kk + 8 (lane / 32) + 0..7 of both operands.  The
// fragments of group kk + 1 are read while group kk's MFMAs run.  One barrier per stage,
// before its last group: by then the stage's last fragments are read, so its slot takes
// the copy S stages ahead, and the last group's MFMAs cover those copies' issue and the
// next stage's first reads.
// Rows past an operand's end read as zero (buffer bounds).

#include "loss.h"

#include "gemm.h"

#include <numeric>
#include <type_traits>

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
// dH and dW products of 4096 tokens x 8192 x 32000 took 2.4 and 2.2 ms.  (m0 is a reserved
// register that the compiler writes right before each use of its own; these kernels have
// none.)
QL_DEV void lload_lds(u32x4 rsrc, int at, int voff, int soff) {
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
// `base`: the tile's first row, `bytes`: from there to the operand's end.  Row r's 16-byte
// chunks sit at chunk ^ f(r), so that the 16 lanes of a read phase (one chunk of 16
// consecutive rows) cover the 64 banks once.
template <int R, int BK>
struct RowOperand {
  static constexpr int kElems = R * BK;
  static constexpr int CH = BK / 8;               // chunks per row
  static constexpr int kRows = 64 / CH;           // rows per 1 KB copy
  static constexpr int kBlocks = R / kRows;       // copies per stage
  static constexpr int kCopies = kBlocks < kWaves ? 1 : kBlocks / kWaves;  // per wave
  static_assert(kCopies == 1 || kCopies % 2 == 0, "a copy's swizzle depends on its parity");
  u32x4 rsrc;
  int voff[2], step;
  int frag, swz;
  static QL_DEV int f(int r) { return (r / (16 / CH)) & (CH - 1); }
  // with fewer copies than waves two waves make the same one: every wave's count of
  // outstanding copies stays the same
  static QL_DEV int block(int wv, int c) { return kBlocks < kWaves ? wv % kBlocks : wv * kCopies + c; }
  QL_DEV void init(const uint16_t *base, int64_t ld, int64_t bytes, int lane, int wv, int first_row) {
    rsrc = lrsrc(base, bytes);
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
  QL_DEV void copy(int at, int wv, int kt_, int c) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_);
    lload_lds(rsrc, at + block(wv, c) * 1024, voff[c & 1], kt * BK * 2 + (c & ~1) * step);
  }
  QL_DEV u32x4 read(const uint16_t *stage, int lane, int t, int kk) const {
    return *reinterpret_cast<const u32x4 *>(stage + frag + t * 32 * BK + (((2 * kk + (lane >> 5)) ^ swz) << 3));
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
  u32x4 rsrc;
  int voff[2], step, stride;
  int frag, unit;
  // rows [0, k) of `base` are within 2^31 bytes (kernels walk longer sums in segments)
  QL_DEV void init(const uint16_t *base, int64_t ld, int64_t bytes, int lane, int wv, int first_col) {
    rsrc = lrsrc(base, bytes);
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
  QL_DEV void copy(int at, int wv, int kt_, int c) const {
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

template <typename F, int... I>
QL_DEV void unrolled(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// acc[i][j] += sum over nk stages of A tile i times B tile j.  A's ring has SA slots and
// B's SB, one after the other at `ring`.
// Stage kt's slots are free after its barrier.  B's copy of stage kt + SB is issued in its
// last group, A's of stage kt + SA in the next stage's groups before the next barrier, so
// the copies are spread: issued at once by all four waves they queue at the address unit
// and hold up the MFMAs behind them.
template <int SA, int SB, int BK, int TA, int TB, typename OpA, typename OpB>
QL_DEV void product(const OpA &A, const OpB &B, uint16_t *ring, int nk, int lane, int wv, f32x16 (&acc)[TA][TB]) {
  constexpr int CA = OpA::kCopies, CB = OpB::kCopies;
  constexpr int NG = BK / 16, NM = TA * TB, NF = TA + TB;  // groups; MFMAs and fragments of each
  constexpr int U = std::lcm(SA, SB);
  // copies that may be in flight at a stage's barrier, where stage kt + 1 has to be whole:
  // those issued after the later of its two
  constexpr int kFly = SB <= SA - 1 ? (SB - 1) * CA + (SB - 2) * CB : (SA - 2) * (CA + CB);
  static_assert(SA > 2 && SB >= 2 && kFly < 64, "ring depths");
  uint16_t *ringb = ring + SA * OpA::kElems;
  const int base = __builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)ring);
  constexpr int kBaseB = SA * OpA::kElems * 2;
  u32x4 fa[2][TA], fb[2][TB];
  auto copy_a = [&](int kt, int slot, int c) { A.copy(base + slot * OpA::kElems * 2, wv, kt, c); };
  auto copy_b = [&](int kt, int slot, int c) { B.copy(base + kBaseB + slot * OpB::kElems * 2, wv, kt, c); };
  auto read = [&](int sa, int sb, int kk, int set, int f) {  // fragment f: A's, then B's
    if (f < TA) fa[set][f] = A.read(ring + sa * OpA::kElems, lane, f, kk);
    else fb[set][f - TA] = B.read(ringb + sb * OpB::kElems, lane, f - TA, kk);
  };
  auto sync = []() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((kFly & 15) | (7 << 4) | ((kFly >> 4) << 14));  // vmcnt(kFly) lgkmcnt(0)
    lbarrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // the first stages, in the order in which the loop issues the later ones
#pragma unroll
  for (int i = -(SA > SB ? SA : SB); i < 0; ++i) {
    if (i - 1 + SA >= 0)
#pragma unroll
      for (int c = 0; c < CA; ++c) copy_a(i - 1 + SA, i - 1 + SA, c);
    if (i + SB >= 0)
#pragma unroll
      for (int c = 0; c < CB; ++c) copy_b(i + SB, i + SB, c);
  }
  sync();
#pragma unroll
  for (int f = 0; f < NF; ++f) read(0, 0, 0, 0, f);
  auto step = [&](auto ic, int kt) {
    constexpr int I = decltype(ic)::value, ia = I % SA, ib = I % SB;
#pragma unroll
    for (int kk = 0; kk < NG; ++kk) {
      const bool last = kk == NG - 1;
      // this group's copies: B's in the last group, a share of A's in the others
      const int c0 = last ? 0 : CA * kk / (NG - 1), c1 = last ? CB : CA * (kk + 1) / (NG - 1);
      // the next group's reads ride on this group's first half, so that they are done by
      // its end
      constexpr int RP = (2 * NF + NM - 1) / NM;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const int i = m / TB, j = m % TB;
        acc[i][j] = lmfma(fa[kk & 1][i], fb[kk & 1][j], acc[i][j]);
#pragma unroll
        for (int f = RP * m; f < RP * (m + 1); ++f)
          if (f < NF) read(last ? (ia + 1) % SA : ia, last ? (ib + 1) % SB : ib, last ? 0 : kk + 1, (kk + 1) & 1, f);
#pragma unroll
        for (int c = c0 + (c1 - c0) * m / NM; c < c0 + (c1 - c0) * (m + 1) / NM; ++c) {
          if (last) copy_b(kt + SB, ib, c);
          else copy_a(kt - 1 + SA, (ia + SA - 1) % SA, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // this wave's copies of stage kt + 1 and its reads of stage kt; with that in every
      // wave, stage kt + 1 is whole and stage kt's slots are free
      if (kk == NG - 2) sync();
    }
  };
  int kt = 0;
  for (; kt + U - 1 < nk; kt += U)
    unrolled([&](auto ic) { step(ic, kt + decltype(ic)::value); }, std::make_integer_sequence<int, U>{});
  unrolled([&](auto ic) { if (kt + decltype(ic)::value < nk) step(ic, kt + decltype(ic)::value); },
           std::make_integer_sequence<int, U - 1>{});
  __builtin_amdgcn_s_waitcnt(0);  // no copy of a stage past the end may still land in LDS
  __syncthreads();
}

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

constexpr int lmax(int a, int b) { return a > b ? a : b; }

// the row of accumulator element v in its 32 x 32 tile
QL_DEV int acc_row(int v, int g) { return 8 * (v >> 2) + 4 * g + (v & 3); }

}  // namespace

// Logits of a tile of BV vocabulary rows x BT tokens, WV x (4 / WV) waves.  The
// vocabulary is on the MFMA's rows, so most of a token's values are in one lane and
// its softmax statistics need one exchange between lanes.
// GRAD false: part[tile][token] = (max, sum of exp(z - max)) over the tile's rows, and
// zlab of the tokens whose label is among them.
// GRAD true: G[token][v] = bf16((exp(z - lse) - [v is the label]) * (dloss / top)).
template <int BV, int BT, int WV, int SA, int SB, int BK, bool GRAD>
__global__ __launch_bounds__(kThreads) void head_logits_kernel(LogitParams p) {
  constexpr int WT = 4 / WV, TA = BV / WV / 32, TB = BT / WT / 32;
  constexpr int kRing = (SA * BV + SB * BT) * BK;  // elements
  constexpr int kLdg = BV + 8;                     // staging of G: [token][BV]
  constexpr int kBytes = lmax(kRing * 2, GRAD ? BT * kLdg * 2 : WV * BT * 8);
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  uint16_t *ring = reinterpret_cast<uint16_t *>(lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  const int tiles_t = (n + BT - 1) / BT;
  if ((int64_t)blockIdx.x >= (int64_t)tiles_t * p.tiles_v) return;
  int tv, tt;
  gemm_tile_of(blockIdx.x, p.tiles_v, tiles_t, 4, tv, tt);
  const int64_t v0 = (int64_t)tv * BV, t0 = (int64_t)tt * BT;
  const int wa = wv / WT * (BV / WV), wb = wv % WT * (BT / WT);  // the wave's first row and column
  RowOperand<BV, BK> A;
  RowOperand<BT, BK> B;
  A.init(p.W + v0 * p.h, p.h, (p.nvoc - v0) * p.h * 2, lane, wv, wa);
  B.init(p.H + t0 * p.h, p.h, ((int64_t)n - t0) * p.h * 2, lane, wv, wb);
  f32x16 acc[TA][TB];
  clear(acc);
  product<SA, SB, BK, TA, TB>(A, B, ring, (int)(p.h / BK), lane, wv, acc);

  const int rows = (int)(p.nvoc - v0 < BV ? p.nvoc - v0 : BV);  // vocabulary rows of this tile
  if constexpr (!GRAD) {
    f32x2 *red = reinterpret_cast<f32x2 *>(lds);  // [WV][BT]
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int64_t t = t0 + wb + 32 * j + l32;
      // the label's row in this tile (none: a row that no lane has)
      const int64_t lab = t < n ? (int64_t)p.label[t] - p.v0 - v0 : -1;
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int row = wa + 32 * i + acc_row(v, g);
          if (row == lab) p.zlab[t] = acc[i][j][v];
          if (row >= rows) acc[i][j][v] = -__builtin_inff();
          mx = fmaxf(mx, acc[i][j][v]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      // a wave whose rows are all past the vocabulary has no maximum: its sum is 0
      const float top = mx == -__builtin_inff() ? 0.0f : mx;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) s += __expf(acc[i][j][v] - top);
      s += __shfl_xor(s, 32, 64);
      if (g == 0) red[wv / WT * BT + wb + 32 * j + l32] = f32x2{mx, s};
    }
    __syncthreads();
    if (threadIdx.x < BT) {
      const int64_t t = t0 + threadIdx.x;
      f32x2 a = red[threadIdx.x];  // rows 0.. of the tile: never empty
#pragma unroll
      for (int w = 1; w < WV; ++w) {
        const f32x2 b = red[w * BT + threadIdx.x];
        const float m = fmaxf(a[0], b[0]);
        a = f32x2{m, a[1] * __expf(a[0] - m) + b[1] * __expf(b[0] - m)};
      }
      if (t < n) p.part[(int64_t)tv * p.ldp + t] = a;
    }
  } else {
    uint16_t *cs = reinterpret_cast<uint16_t *>(lds);
    const float top = *p.top;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int col = wb + 32 * j + l32;
      const int64_t t = t0 + col;
      const bool live = t < n;
      const float lse = live ? p.lse[t] : 0.0f, dl = live && top > 0.0f ? p.dloss[t] / top : 0.0f;
      const int64_t lab = live ? (int64_t)p.label[t] - p.v0 - v0 : -1;
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = wa + 32 * i + 8 * q + 4 * g + e;
            const float pr = __expf(acc[i][j][4 * q + e] - lse);
            o[e] = row < rows ? (row == lab ? pr - 1.0f : pr) * dl : 0.0f;
          }
          *reinterpret_cast<u32x2 *>(cs + col * kLdg + wa + 32 * i + 8 * q + 4 * g) =
              u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        }
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < BT * BV / 8; ch += kThreads) {
      const int col = ch / (BV / 8), c8 = ch % (BV / 8);
      if (t0 + col < n)
        *reinterpret_cast<u32x4 *>(p.G + (t0 + col) * p.ldg + v0 + c8 * 8) =
            *reinterpret_cast<const u32x4 *>(cs + col * kLdg + c8 * 8);
    }
  }
}

// dH partial sums: part[split][token][k] (+)= sum over the split's vocabulary entries v
// of G[token][v] W[v][k].  G's columns past the piece are zero and W's rows past it read
// as zero, so the last step may be short.
template <int BM, int SA, int SB, int BK>
__global__ __launch_bounds__(kThreads) void head_dh_kernel(HeadGradParams p) {
  constexpr int BN = 256, WM = BM == 256 ? 2 : 1, WN = 4 / WM;
  constexpr int TA = BM / WM / 32, TB = BN / WN / 32;
  __shared__ __attribute__((aligned(16))) uint16_t ring[(SA * BM + SB * BN) * BK];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  const int tiles_m = (n + BM - 1) / BM;
  if ((int)blockIdx.x >= tiles_m * p.tiles_n) return;
  int tm, tn;
  gemm_tile_of(blockIdx.x, tiles_m, p.tiles_n, 4, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int64_t k0 = (int64_t)blockIdx.y * p.kper;
  const int64_t k1 = k0 + p.kper < p.nvoc ? k0 + p.kper : p.nvoc;
  const int wa = wv / WN * (BM / WM), wb = wv % WN * (BN / WN);
  RowOperand<BM, BK> A;
  ColOperand<BN, BK> B;
  f32x16 acc[TA][TB];
  clear(acc);
  const int64_t seg = col_segment(p.h);
  for (int64_t k = k0; k < k1; k += seg) {
    const int64_t len = k1 - k < seg ? k1 - k : seg;
    A.init(p.G + m0 * p.ldg + k, p.ldg, ((int64_t)n - m0) * p.ldg * 2 - k * 2, lane, wv, wa);
    B.init(p.W + k * p.h + n0, p.h, (p.nvoc - k) * p.h * 2 - n0 * 2, lane, wv, wb);
    product<SA, SB, BK, TA, TB>(A, B, ring, (int)((len + BK - 1) / BK), lane, wv, acc);
  }
  float *out = p.part + (int64_t)blockIdx.y * p.rows * p.h;
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t m = m0 + wa + 32 * i + acc_row(v, g), c = n0 + wb + 32 * j + l32;
        if (m >= n || c >= p.h) continue;
        float *dst = out + m * p.h + c;
        *dst = p.add ? *dst + acc[i][j][v] : acc[i][j][v];
      }
}

// dW[v][k] = bf16(top * sum over the tokens of G[token][v] H[token][k]).
template <int SA, int SB, int BK>
__global__ __launch_bounds__(kThreads) void head_dw_kernel(HeadGradParams p) {
  constexpr int BM = 256, BN = 256, TA = 4, TB = 4, kLdc = BN + 8;
  constexpr int kBytes = lmax((SA * BM + SB * BN) * BK * 2, BM * kLdc * 2);
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  uint16_t *ring = reinterpret_cast<uint16_t *>(lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  int tm, tn;
  gemm_tile_of(blockIdx.x, p.tiles_m, p.tiles_n, 4, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wa = wv / 2 * 128, wb = wv % 2 * 128;
  ColOperand<BM, BK> A;
  ColOperand<BN, BK> B;
  f32x16 acc[TA][TB];
  clear(acc);
  const int64_t seg = col_segment(p.h > p.ldg ? p.h : p.ldg);
  for (int64_t k = 0; k < n; k += seg) {
    const int64_t len = n - k < seg ? n - k : seg;
    A.init(p.G + k * p.ldg + m0, p.ldg, (n - k) * p.ldg * 2 - m0 * 2, lane, wv, wa);
    B.init(p.H + k * p.h + n0, p.h, (n - k) * p.h * 2 - n0 * 2, lane, wv, wb);
    product<SA, SB, BK, TA, TB>(A, B, ring, (int)((len + BK - 1) / BK), lane, wv, acc);
  }
  uint16_t *cs = reinterpret_cast<uint16_t *>(lds);
  const float top = n > 0 ? *p.top : 0.0f;
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        cs[(wa + 32 * i + acc_row(v, g)) * kLdc + wb + 32 * j + l32] =
            (uint16_t)(pack_bf16x2(top * acc[i][j][v], 0.0f) & 0xFFFFu);
  __syncthreads();
  for (int ch = threadIdx.x; ch < BM * BN / 8; ch += kThreads) {
    const int row = ch / (BN / 8), c8 = ch % (BN / 8);
    const int64_t m = m0 + row, c = n0 + c8 * 8;
    if (m < p.nvoc && c < p.h)
      *reinterpret_cast<u32x4 *>(p.dW + m * p.h + c) = *reinterpret_cast<const u32x4 *>(cs + row * kLdc + c8 * 8);
  }
}

namespace {
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }
}  // namespace

int logit_tile_v(int64_t max_tokens) { return max_tokens <= 128 ? 128 : 256; }

hipError_t launch_logit_stats(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  p.tiles_v = (int)cdiv(p.nvoc, logit_tile_v(max_tokens));
  if (max_tokens <= 32) return launch(head_logits_kernel<128, 32, 4, 4, 4, 64, false>, (unsigned)p.tiles_v, kThreads, st, p);
  if (max_tokens <= 128)
    return launch(head_logits_kernel<128, 128, 2, 3, 2, 64, false>, (unsigned)p.tiles_v, kThreads, st, p);
  return launch(head_logits_kernel<256, 256, 2, 3, 2, 64, false>, (unsigned)(p.tiles_v * cdiv(max_tokens, 256)), kThreads, st,
                p);
}

hipError_t launch_logit_grad(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  if (max_tokens <= 32) {
    p.tiles_v = (int)cdiv(p.nvoc, 128);
    return launch(head_logits_kernel<128, 32, 4, 4, 4, 64, true>, (unsigned)p.tiles_v, kThreads, st, p);
  }
  if (max_tokens <= 128) {
    p.tiles_v = (int)cdiv(p.nvoc, 128);
    return launch(head_logits_kernel<128, 128, 2, 3, 2, 64, true>, (unsigned)p.tiles_v, kThreads, st, p);
  }
  p.tiles_v = (int)cdiv(p.nvoc, 256);
  return launch(head_logits_kernel<256, 256, 2, 3, 2, 64, true>, (unsigned)(p.tiles_v * cdiv(max_tokens, 256)), kThreads, st,
                p);
}

hipError_t launch_head_dh(HeadGradParams &p, int splits, int64_t max_tokens, hipStream_t st) {
  p.tiles_n = (int)cdiv(p.h, 256);
  if (max_tokens <= 64)
    return launch(head_dh_kernel<64, 3, 2, 64>, dim3((unsigned)(cdiv(max_tokens, 64) * p.tiles_n), (unsigned)splits), kThreads,
                  st, p);
  return launch(head_dh_kernel<256, 3, 2, 64>, dim3((unsigned)(cdiv(max_tokens, 256) * p.tiles_n), (unsigned)splits), kThreads,
                st, p);
}

hipError_t launch_head_dw(HeadGradParams &p, hipStream_t st) {
  p.tiles_m = (int)cdiv(p.nvoc, 256);
  p.tiles_n = (int)cdiv(p.h, 256);
  return launch(head_dw_kernel<5, 5, 32>, (unsigned)(p.tiles_m * p.tiles_n), kThreads, st, p);
}

}  // namespace ql
