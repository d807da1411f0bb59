// The products of the output head's cross entropy for few tokens, for gfx950: logits on
// 128 x 32 and 128 x 128 tiles, dH for at most 64 tokens.  They are bound by reading the
// head once.  (More tokens, and dW: loss_wide.hip.)
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
// 16 tokens of 4096 values, 32000 words (262 MB): logits 41 us where the head is partly in
// the last-level cache, 50 to 62 from memory, as long as a plain read of it plus the start
// and the softmax (deeper rings: no faster); dH 60 us.

#include "loss_tiles.h"

#include "gemm.h"

#include <numeric>
#include <type_traits>

namespace ql {
namespace {

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
QL_DEV void product(const OpA &A, const OpB &B, const u32x4 &ra, const u32x4 &rb, uint16_t *ring, int nk, int lane,
                    int wv, f32x16 (&acc)[TA][TB]) {
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
  auto copy_a = [&](int kt, int slot, int c) { A.copy(ra, base + slot * OpA::kElems * 2, wv, kt, c); };
  auto copy_b = [&](int kt, int slot, int c) { B.copy(rb, base + kBaseB + slot * OpB::kElems * 2, wv, kt, c); };
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

constexpr int lmax(int a, int b) { return a > b ? a : b; }

}  // namespace

// Logits of a tile of BV vocabulary rows x BT tokens, WV x (4 / WV) waves.  The
// vocabulary is on the MFMA's rows, so most of a token's values are in one lane and
// its softmax statistics need one exchange between lanes.
// GRAD false: part[tile][token] = (max, sum of exp(z - max)) over the tile's rows, and
// zlab of the tokens whose label is among them.
// GRAD true: G[token][v] = bf16((exp(z - lse) - [v is the label]) * (dloss / top)).
// FEW (statistics only): the tokens are at most BT, one tile with or without those that
// carry no loss, so they come straight from H and no list is made.  (A token is a column
// of the product: what the others' rows hold stays in their own statistics, which nobody
// reads.)  16 x 4096 x 32000: 63 us in all, with a list and a copy of the rows first 69.
// ONCE: the head is read past the caches (launch_logit_stats_few).
template <int BV, int BT, int WV, int SA, int SB, int BK, bool GRAD, bool FEW, bool ONCE>
__global__ __launch_bounds__(kThreads) void head_logits_kernel(LogitParams p) {
  constexpr int WT = 4 / WV, TA = BV / WV / 32, TB = BT / WT / 32;
  constexpr int kRing = (SA * BV + SB * BT) * BK;  // elements
  constexpr int kLdg = BV + 8;                     // staging of G: [token][BV]
  constexpr int kBytes = lmax(kRing * 2, GRAD ? BT * kLdg * 2 : WV * BT * 8);
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  uint16_t *ring = reinterpret_cast<uint16_t *>(lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  static_assert(!FEW || (!GRAD && BT == kFewTokens), "one tile of tokens");
  const int n = FEW ? (int)p.M : *p.count;
  int64_t few_label = -1;
  if constexpr (FEW) few_label = l32 < n ? p.labels[l32] : -1;
  const int tiles_t = (n + BT - 1) / BT;
  if ((int64_t)blockIdx.x >= (int64_t)tiles_t * p.tiles_v) return;
  int tv, tt;
  gemm_tile_of(blockIdx.x, p.tiles_v, tiles_t, 4, tv, tt);
  const int64_t v0 = (int64_t)tv * BV, t0 = (int64_t)tt * BT;
  const int wa = wv / WT * (BV / WV), wb = wv % WT * (BT / WT);  // the wave's first row and column
  RowOperand<BV, BK, ONCE> A;
  std::conditional_t<FEW, RowOperand<BT, BK>, BlockRows<BT, BK>> B;
  A.init(p.h, lane, wv, wa);
  B.init(FEW ? p.h : p.h * 64, lane, wv, wb);
  const u32x4 ra = lrsrc(p.W + v0 * p.h, (p.nvoc - v0) * p.h * 2);
  const u32x4 rb = lrsrc(p.H + t0 * p.h, ((FEW ? n : (n + 31) / 32 * 32) - t0) * p.h * 2);
  f32x16 acc[TA][TB];
  clear(acc);
  product<SA, SB, BK, TA, TB>(A, B, ra, rb, ring, (int)(p.h / BK), lane, wv, acc);

  const int rows = (int)(p.nvoc - v0 < BV ? p.nvoc - v0 : BV);  // vocabulary rows of this tile
  if constexpr (!GRAD) {
    f32x2 *red = reinterpret_cast<f32x2 *>(lds);  // [WV][BT]
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int64_t t = t0 + wb + 32 * j + l32;
      // the label's row in this tile (none: a row that no lane has)
      const int64_t lab = FEW ? few_label - v0 : t < n ? (int64_t)p.label[t] - p.v0 - v0 : -1;
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
      f32x2 a = red[threadIdx.x];
#pragma unroll
      for (int w = 1; w < WV; ++w) {
        const f32x2 b = red[w * BT + threadIdx.x];
        const float m = fmaxf(a[0], b[0]);
        const float ref = m == -__builtin_inff() ? 0.0f : m;  // both waves' words masked: the sum is 0
        a = f32x2{m, a[1] * __expf(a[0] - ref) + b[1] * __expf(b[0] - ref)};
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
      const float lse = live ? p.lse[t] : 0.0f;
      const float raw = live ? p.dloss[t] : 0.0f, dl = top > 0.0f ? raw / top : raw;
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
      const int col = ch / (BV / 8), c8 = ch % (BV / 8);  // tokens past the last: zero, within a whole 32
      *reinterpret_cast<u32x4 *>(p.G + blocked(t0 + col, v0 + c8 * 8, p.gblocks)) =
          *reinterpret_cast<const u32x4 *>(cs + col * kLdg + c8 * 8);
    }
  }
}

// dH partial sums for at most 64 tokens: part[split][token][k] (+)= sum over the split's vocabulary entries v
// of G[token][v] W[v][k].  G's columns past the piece are zero and W's rows past it read
// as zero, so the last step may be short.
__global__ __launch_bounds__(kThreads) void head_dh_kernel(HeadGradParams p) {
  constexpr int BM = 64, BN = 256, TA = 2, TB = 2, SA = 3, SB = 2, BK = 64;
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
  const int wa = 0, wb = wv * 64;
  BlockRows<BM, BK> A;
  ColOperand<BN, BK> B;
  A.init(p.gblocks * 2048, lane, wv, wa);
  B.init(p.h, lane, wv, wb);
  f32x16 acc[TA][TB];
  clear(acc);
  const int64_t seg = col_segment(p.h);
  for (int64_t k = k0; k < k1; k += seg) {
    const int64_t len = k1 - k < seg ? k1 - k : seg;
    const u32x4 ra = lrsrc(p.G + (k >> 5) * 1024, (n + 31) / 32 * p.gblocks * 2048 - (k >> 5) * 2048);
    const u32x4 rb = lrsrc(p.W + k * p.h + n0, (p.nvoc - k) * p.h * 2 - n0 * 2);
    product<SA, SB, BK, TA, TB>(A, B, ra, rb, ring, (int)((len + BK - 1) / BK), lane, wv, acc);
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

namespace {
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }
}  // namespace

// Whether the logits run on 256 x 256 tiles, one persistent workgroup per compute unit, or
// on 128 x 128, two workgroups per compute unit: the larger ones once the smaller ones take
// a second round (more than 512), before which they would leave compute units idle (4096
// values, 256 tokens: 10000 words 92 against 46 us, 32000 words 101 against 93, 50257 words,
// 786 small tiles, 136 against 164).  Up to 128 tokens half of every larger tile would be
// empty; and they need h of three 64-deep stages.
bool logits_wide(int64_t max_tokens, int64_t h, int64_t nvoc) {
  return max_tokens > 128 && h >= 192 && cdiv(max_tokens, 128) * cdiv(nvoc, 128) > 512;
}
int logit_parts(int64_t max_tokens, int64_t h, int64_t V) {
  return logits_wide(max_tokens, h, V) ? 2 * (int)cdiv(V, 256) : (int)cdiv(V, 128);
}

namespace {
template <bool GRAD>
hipError_t logits(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  if (logits_wide(max_tokens, p.h, p.nvoc)) return launch_logit_wide(p, GRAD, st);
  // G is written (zero past the piece) up to a multiple of 256
  p.tiles_v = GRAD ? 2 * (int)cdiv(p.nvoc, 256) : (int)cdiv(p.nvoc, 128);
  if constexpr (GRAD)
    if (max_tokens <= kFewTokens)
      return launch(head_logits_kernel<128, 32, 4, 4, 4, 64, true, false, false>, (unsigned)p.tiles_v, kThreads, st, p);
  // A launch holds fewer than 2^32 threads.  Only statistics of h below 192 get there (131072
  // tokens, 2^21 words: 2^24 workgroups): the vocabulary then takes several launches.
  const int64_t tiles_t = cdiv(max_tokens, 128), most = (((int64_t)1 << 24) - 1) / tiles_t;
  const int tiles_v = p.tiles_v;
  for (int64_t first = 0; first < tiles_v; first += most) {
    LogitParams q = p;
    q.W += 128 * first * p.h, q.v0 += 128 * first, q.nvoc -= 128 * first;
    if constexpr (!GRAD) q.part += first * p.ldp;
    q.tiles_v = (int)(tiles_v - first < most ? tiles_v - first : most);
    const hipError_t e = launch(head_logits_kernel<128, 128, 2, 3, 2, 64, GRAD, false, false>,
                                (unsigned)(q.tiles_v * tiles_t), kThreads, st, q);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
}  // namespace

hipError_t launch_logit_stats(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  return logits<false>(p, max_tokens, st);
}
hipError_t launch_logit_stats_few(LogitParams &p, hipStream_t st) {
  p.tiles_v = (int)cdiv(p.nvoc, 128);
  // A head larger than the last-level cache is read past it, which frees the way to memory
  // (4096 values: 64000 words 105 -> 99 us; 8192 x 128256 462 -> 393 us).  A smaller one may
  // still be there from the call before, and reading it past the cache then costs more than
  // it gains where it is not.  Whole calls of 16 tokens, 4096 x 32000: the same head again 44
  // us, past the cache 65; eleven heads in turn, each from memory, 67 and 62.  4096 x 16384:
  // 25 and 36; 39 and 37.
  if (p.nvoc * p.h * 2 > ((int64_t)1 << 28))
    return launch(head_logits_kernel<128, 32, 4, 4, 4, 64, false, true, true>, (unsigned)p.tiles_v, kThreads, st, p);
  return launch(head_logits_kernel<128, 32, 4, 4, 4, 64, false, true, false>, (unsigned)p.tiles_v, kThreads, st, p);
}
hipError_t launch_logit_grad(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  return logits<true>(p, max_tokens, st);
}

hipError_t launch_head_dh(HeadGradParams &p, int64_t max_tokens, hipStream_t st) {
  if (max_tokens > 64) return launch_head_dh_wide(p, st);
  p.tiles_n = (int)cdiv(p.h, 256);
  return launch(head_dh_kernel, dim3((unsigned)p.tiles_n, (unsigned)cdiv(p.nvoc, p.kper)), kThreads, st, p);
}

}  // namespace ql
