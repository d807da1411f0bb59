// Attention of packed tokens backward, for gfx950.  With the forward's lse,
//   p = exp(z - lse),  D_i = dO_i . O_i,  dP = dO V^T
//   dS = p (dP - D) (times 1 - tanh^2 of a capped score)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = p^T dO
// dK and dV of a key head sum over the query heads that share it.  Two kernels, each the
// only writer of its outputs, so that nothing is added atomically and results repeat; the
// price is that z and dP are formed in both: seven products instead of five.
//
//   attn_dq   128 queries of a head per workgroup, a wave 32 in its lanes, as the forward.
//             It also leaves D, lse in units of log2 and the reach of every 32 queries'
//             spans in the workspace for
//   attn_dkv  128 keys of a key head per workgroup, a wave 32 in its lanes with their dK and
//             dV in registers, over the tiles of 32 queries that see any of them, of every
//             query head of the group.  The keys are a wave's second operand in registers;
//             the values are read from LDS each time: both in registers leave none for reads
//             ahead (307 us for 2048 tokens and 64 heads; p in one wave and dS in another,
//             through LDS, 205 us).
// p and dS are rounded to bf16 as operands of the products that follow.
//
// Bound by the matrix cores, the weights' vector operations beside them and the waits between
// dependent products: two waves fit a SIMD at the 224 to 251 registers that dQ takes at 128
// values and the 253 to 256 of dK and dV (up to 10 more are spilled, none within the plain form's
// products); at 64 values 148 to 188 let a unit hold one workgroup of eight waves or, except
// capped ones, three of four.  Measured, causal, heads of 128: 2048 tokens of 64 heads dQ 119
// to 148 us, dK and dV 149 to 195 (the clock falls; 0.94 PFLOP/s by the seven products, matrix
// cores busy 42 % of the cycles, no bank conflicts); 4001 tokens in 9 documents, 32 heads for 8,
// dQ 94, dK and dV 150 and their sum 12.  No gain: raised priority for the weights' phase, as
// the forward has.
//
// D from the forward's bf16 O is off by a rounding of O, which all of a row's dS share: with
// few keys, whose dS nearly cancel, that would be percents of dQ.  Queries that see at most
// 256 keys, or whose head's bias leaves weight to a few tens (1531 tokens, heads biased by 0.5 a
// token: dQ off by 0.0028 of its norm, so 0.0024), have D = sum_j p_ij dP_ij in a pass of its own
// over the keys of such queries instead.  Which one is a query's own matter: what else is in its
// workgroup changes nothing.

#include "attn_tiles.h"

namespace ql {
namespace {

constexpr int kRowsWg = 128;  // queries per workgroup
constexpr int kKeysWg = 128;  // keys per workgroup
constexpr int kTile = 64;     // keys per tile of attn_dq
constexpr int kRows = 32;     // queries per tile of attn_dkv
// attn_dq's passes: D by its own sum; dQ; dQ where what is not finite is looked for
enum { kOwnD, kSums, kCarefulSums };
constexpr int kFewKeys = 256;
constexpr float kSteep = 1.0f / 16;  // of a bias, towards a query's own key or away from it

struct BwdWork {
  f32x2 *stat;  // [hq][ld] lse in units of log2, and D
  int4 *reach;  // [ld / 32]: union and intersection of 32 rows' spans
  int64_t ld;   // M rounded up to 128
  float *part;  // splits > 1: dK, then dV, of each split, [splits][M][hk][d]
  int splits, groups;  // of a key's sum over the queries: workgroups, and groups of waves in each
  int heads;           // of the splits, those by query heads; the rest are by tiles
};

inline int64_t padded(int64_t M) { return (M + 127) / 128 * 128; }

// Parts of a key's sum over the queries: few key heads and tokens leave compute units without
// a workgroup, or with one long one.  Two parts are two groups of waves of one workgroup, with
// the even and the odd tiles, joined through LDS; more are workgroups of two each, which share
// out the query heads and, where these are too few, the tiles (33 tokens, 64 heads for one: by
// tiles alone 142 us, so 32).  Their sums go through the workspace in the time of six tiles.
// So a part keeps 4 tiles up to two parts for each unit, 16 up to four, and 128 beyond,
// where long documents' workgroups need not wait for longer ones.  Backward in us, in 1, 2, 4,
// 8, 16 and 32 parts by tiles, 128 values a head (64 take the same rule):
//   tokens  heads  key heads   of 128 keys
//     512     32       8          32       111,   80,   63,  52,  51,  71
//    2048      8       1          16       682,  462,  264, 165, 118,  97
//    2048      8       8         128       133,  106,   94, 100, 135, 200
//    2048     32       8         128       386,  275,  192, 171, 211, 292
//    2048     32      32         512       166,  153,  203
//    2048     64      64        1024       270,  286
//    4001     32       8         256       803,  602,  473, 504 (in a window of 450, where fewer tiles
//                                          186,  153,  182, 215  are seen than is known here: 4)
//    8192      8       1          64      2678, 1806, 1005, 626, 488, 532
inline int bwd_parts(int64_t M, int64_t hq, int64_t hk) {
  const int64_t units = (M + kKeysWg - 1) / kKeysWg * hk, rows = (M + kRows - 1) / kRows, tiles = rows * (hq / hk);
  int s = 1;
  while (s < 32 && s < rows * (hq / hk) && units * s < 2048 && tiles >= (units * s < 512 ? 8 : units * s < 1024 ? 32 : 256) * s)
    s *= 2;
  return s;
}

inline BwdWork bwd_work(int64_t M, int64_t hq, int64_t hk, void *ws) {
  const int64_t ld = padded(M);
  f32x2 *stat = reinterpret_cast<f32x2 *>(ws);
  int4 *reach = reinterpret_cast<int4 *>(stat + hq * ld);
  const int parts = bwd_parts(M, hq, hk), groups = parts > 1 ? 2 : 1, splits = parts / groups;
  int heads = 1;
  while (heads < splits && 2 * heads <= hq / hk) heads *= 2;
  return BwdWork{stat, reach, ld, reinterpret_cast<float *>(reach + ld / 32), splits, groups, heads};
}

}  // namespace

// KG: groups of four waves, each with every KG-th tile of keys, as in the forward.
template <int D, Form FORM, int KG>
__global__ __launch_bounds__(kThreads * KG, 2) void attn_dq_kernel(AttnArgs a, AttnGrads gr, BwdWork w) {
  __shared__ __attribute__((aligned(1024))) uint16_t ring[KG][4 * kTile * D];  // K, V; two slots
  __shared__ int ends[4 * kWaves], spoiled[kWaves * KG];
  __shared__ float owns[KG][kWaves][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wave / kWaves, wv = wave % kWaves;
  const int g = lane >> 5, l32 = lane & 31;
  const int tiles = (int)((a.M + kRowsWg - 1) / kRowsWg);
  int place, head;
  unit_place(blockIdx.x, tiles, a.hq, place, head);
  const int64_t q0 = (int64_t)(tiles - 1 - place) * kRowsWg;
  const int64_t row = q0 + 32 * wv + l32;
  const bool live = row < a.M;
  const int hk = head / (a.hq / a.hk);
  const Span span = span_of(a.spans, row, a.M);
  const Reach reach = reach_of(span);
  const bool any = span.lo < span.hi;
  const float slope2 = FORM != kPlain && a.slopes ? a.slopes[head] * kLog2e : 0.0f;
  // whether this query has D by its own sum, and the keys of the wave's that do
  const bool sums = any && (span.hi - span.lo <= kFewKeys || (FORM != kPlain && __builtin_fabsf(slope2) >= kSteep * kLog2e));
  const int own_lo = rows_min(sums ? span.lo : 0x7FFFFFFF), own_hi = rows_max(sums ? span.hi : 0);
  if (kg == 0 && lane == 0) {
    ends[wv] = reach.lo, ends[kWaves + wv] = reach.hi;
    ends[2 * kWaves + wv] = own_lo, ends[3 * kWaves + wv] = own_hi;
  }
  u32x4 qf[D / 16], df[D / 16];
  load_rows<D>(qf, a.Q + row * a.ldq + (int64_t)head * a.d, live, a.d, g);
  load_rows<D>(df, gr.dO + (row * a.hq + head) * a.d, live, a.d, g);
  float delta = 0.0f, lse2 = 0.0f;
  {
    u32x4 of[D / 16];
    load_rows<D>(of, gr.O + (row * a.hq + head) * a.d, live, a.d, g);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        delta = __builtin_fmaf(bf16_lo(df[kk][i]), bf16_lo(of[kk][i]),
                               __builtin_fmaf(bf16_hi(df[kk][i]), bf16_hi(of[kk][i]), delta));
    delta = both_halves_sum(delta);
    if (live) lse2 = gr.lse[(int64_t)head * a.M + row] * kLog2e;
    // rows that see nothing (and those past the last) carry no gradient
    if (!any) delta = 0.0f, lse2 = __builtin_inff();
    // where rows are summed over, one that sees nothing, or is past the last, has to be masked: no
    // key is seen by all
    const bool gap = __any(!any);
    if (head == 0 && kg == 0 && lane == 0)
      w.reach[row >> 5] = int4{reach.lo, reach.hi, gap ? 0x7FFFFFFF : reach.all_lo, reach.all_hi};
  }
  __syncthreads();
  // the workgroup's: least and most over the waves; nothing is seen: 0 to 0 (the least was INT_MAX)
  auto from_to = [&](const int *lo, const int *hi, int &first, int &last) {
    first = lo[0], last = hi[0];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) {
      first = lo[v] < first ? lo[v] : first;
      last = hi[v] > last ? hi[v] : last;
    }
    first = __builtin_amdgcn_readfirstlane(first < last ? first : last);
    last = __builtin_amdgcn_readfirstlane(last);
  };
  int first, last;
  from_to(ends, ends + kWaves, first, last);

  f32x16 acc[D / 32];
  const float c = a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e, in2 = a.cap > 0.0f ? 2.0f * c / a.cap : 0.0f;
  constexpr int kTileBytes = kTile * D * 2;
  Tile<D, true> tk, tv;
  tk.init((uint32_t)a.ldk * 2, (uint32_t)a.d * 2, lane, wv);
  tv.init((uint32_t)a.ldv * 2, (uint32_t)a.d * 2, lane, wv);
  TileSource sk, sv;
  sk.init(a.K, a.ldk, hk, a.d, a.M);
  sv.init(a.V, a.ldv, hk, a.d, a.M);
  const int base = lds_address(ring[kg]);
  Reader<D> read;
  read.init(lane);
  auto fetch = [&](int k0, int slot) {
    sk.copy(tk, k0, base + slot * kTileBytes, wv);
    sv.copy(tv, k0, base + (2 + slot) * kTileBytes, wv);
  };
  float own = 0.0f;  // D by its sum, of this lane half's keys
  auto step = [&](int k0, int slot, bool masked, auto pass) {
    constexpr bool kSum = decltype(pass)::value == kOwnD, kCareful = decltype(pass)::value == kCarefulSums;
    const uint32_t kt = base + slot * kTileBytes, vt = kt + 2 * kTileBytes;
    const uint32_t kr = kt + read.row, vr = vt + read.row, kc = kt + read.col;
    const int from = span.lo - k0 - 4 * g, width = span.hi - span.lo;
    const float away = (float)(k0 + 4 * g - (int)row);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x16 z[2];  // scores; dP
      zero(z);
      constexpr int kGroups = D / 16, kAhead = 2;
      u32x4 f[kAhead + 1][2];
      auto rows = [&](int n) {
        f[n % (kAhead + 1)][0] = row_frag<D>(kr, t, n);
        f[n % (kAhead + 1)][1] = row_frag<D>(vr, t, n);
      };
#pragma unroll
      for (int n = 0; n < kAhead; ++n) rows(n);
#pragma unroll
      for (int kk = 0; kk < kGroups; ++kk) {
        if (kk + kAhead < kGroups) rows(kk + kAhead);
        z[0] = lmfma(f[kk % (kAhead + 1)][0], qf[kk], z[0]);
        z[1] = lmfma(f[kk % (kAhead + 1)][1], df[kk], z[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (FORM == kCapped) tanh_all(reinterpret_cast<f32x16(&)[1]>(z[0]), in2);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int j = 32 * t + acc_row(v, 0);
        float p, slack = 1.0f;
        if constexpr (FORM != kPlain) {
          const float x = z[0][v] * (FORM == kCapped ? cap2 : c);
          if constexpr (FORM == kCapped) slack = 1.0f - z[0][v] * z[0][v];
          p = __builtin_amdgcn_exp2f(__builtin_fmaf(-slope2, __builtin_fabsf(away + (float)j), x) - lse2);
        } else {
          p = __builtin_amdgcn_exp2f(__builtin_fmaf(z[0][v], c, -lse2));
        }
        z[1][v] = p * (z[1][v] - (kSum ? 0.0f : delta));
        if constexpr (FORM == kCapped && !kSum) z[1][v] *= slack;
      }
      if (masked)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int j = 32 * t + acc_row(v, 0);
          z[1][v] = j < from || j - from >= width ? 0.0f : z[1][v];
        }
      if constexpr (kSum) {
#pragma unroll
        for (int v = 0; v < 16; ++v) own += z[1][v];
        continue;
      }
      const u32x4 ds[2] = {pack8(z[1], 0), pack8(z[1], 1)};
      constexpr int kTiles = D / 32, kColsAhead = 3;
      if constexpr (kCareful) {
#pragma unroll
        for (int i = 0; i < 2 * kTiles; ++i) {
          u32x4 k = col_frag<D>(kc, i % kTiles, 2 * t + i / kTiles);
          if (masked) k = finite(k);
          acc[i % kTiles] = lmfma(k, ds[i / kTiles], acc[i % kTiles]);
          __builtin_amdgcn_sched_barrier(0);
        }
        continue;
      }
      u32x4 w[kColsAhead + 1];
#pragma unroll
      for (int n = 0; n < kColsAhead; ++n) w[n] = col_frag<D>(kc, n % kTiles, 2 * t + n / kTiles);
#pragma unroll
      for (int i = 0; i < 2 * kTiles; ++i) {
        const int n = i + kColsAhead;
        if (n < 2 * kTiles) w[n % (kColsAhead + 1)] = col_frag<D>(kc, n % kTiles, 2 * t + n / kTiles);
        acc[i % kTiles] = lmfma(w[i % (kColsAhead + 1)], ds[i / kTiles], acc[i % kTiles]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (kCareful)
      if (masked)
        for (uint64_t odd = odd_rows<D, kTile>(kt, lane); odd; odd &= odd - 1) {
          const int r = (int)__builtin_ctzll(odd);
          spoil<D>(acc, kt, r, k0 + r >= span.lo && k0 + r < span.hi, g);
        }
  };
  auto walk = [&](auto pass, int first, int last, int lo, int hi) {  // the workgroup's keys, the wave's
    int slot = 0;
    if (first + kg * kTile < last) fetch(first + kg * kTile, 0);
    for (int at = first; at < last; at += KG * kTile, slot ^= 1) {
      const int k0 = at + kg * kTile;
      tile_sync();
      if (k0 + KG * kTile < last) fetch(k0 + KG * kTile, slot ^ 1);
      if (k0 >= hi || k0 + kTile <= lo) continue;
      step(k0, slot, k0 < reach.all_lo || k0 + kTile > reach.all_hi, pass);
    }
  };
  int own_first, own_last;
  from_to(ends + 2 * kWaves, ends + 3 * kWaves, own_first, own_last);
  if (own_first < own_last) {
    walk(std::integral_constant<int, kOwnD>{}, own_first, own_last, own_lo, own_hi);
    own = both_halves_sum(own);
    if constexpr (KG > 1) {
      owns[kg][wv][lane] = own;
      tile_sync();
      own = owns[0][wv][lane] + owns[1][wv][lane];
    }
    if (sums) delta = own;
    tile_sync();  // the last tile is read
  }
  if (kg == 0 && g == 0) w.stat[head * w.ld + row] = f32x2{lse2, delta};
  zero(acc);
  walk(std::integral_constant<int, kSums>{}, first, last, reach.lo, reach.hi);
  // (as in the forward: taken again if what masked keys hold has spoiled a sum)
  if (any_wave(any && !all_finite(acc), spoiled, wave, kWaves * KG)) {
    zero(acc);
    walk(std::integral_constant<int, kCarefulSums>{}, first, last, reach.lo, reach.hi);
  }
  if constexpr (KG > 1) {
    static_assert(KG == 2, "one group's sums go to the other");
    f32x4 *join = reinterpret_cast<f32x4 *>(ring) + wv * (D / 8 * 64) + lane;
    __syncthreads();  // the last tiles are read
    if (kg == 1) {
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          join[64 * (4 * t + q)] = f32x4{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
    }
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 x = join[64 * (4 * t + q)];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][4 * q + i] += x[i];
      }
  }
  store_row<D>(gr.dQ + (row * a.hq + head) * a.d, acc, any ? a.scale : 0.0f, live, a.d, g);
}

template <int D, int KG>
struct DkvLds {
  // (tiles begin at multiples of 1 KB)
  uint16_t v[kKeysWg * D];
  union {
    uint16_t rows[KG][2][2][kRows * D];             // a group's Q and dO; two slots
    f32x4 join[KG > 1 ? kWaves : 1][D / 8][kWave];  // the second group's sums, dK's and then dV's
  };
  f32x2 stat[KG][2][kRows];
  int span[KG][2][2 * kRows];
  int spoiled[kWaves * KG];
};

// Row `dst` of a split's sums from accumulators whose columns are rows.
template <int D>
QL_DEV void store_sums(float *dst, const f32x16 (&acc)[D / 32], bool live, int d, int g) {
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y = acc[e][4 * q + i];
        asm volatile("" : "+v"(y));  // a copy: taken as it is, the loop's accumulators are split for it and spill
        x[i] = y;
      }
      const int i = 32 * e + 8 * q + 4 * g;
      if (live && i < d) *reinterpret_cast<f32x4 *>(dst + i) = x;
    }
}

// The second group's sums onto the first's.
template <int D>
QL_DEV void join_groups(f32x16 (&x)[D / 32], f32x4 (&at)[D / 8][kWave], int kg, int lane) {
  if (kg == 1) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = x[e][4 * q + i];
          asm volatile("" : "+v"(v));  // (a copy, as in store_sums)
          y[i] = v;
        }
        at[4 * e + q][lane] = y;
      }
  }
  __syncthreads();
  if (kg == 0)
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 y = at[4 * e + q][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[e][4 * q + i] += y[i];
      }
  __syncthreads();
}

// SPLIT: one of several workgroups of these keys, whose sums go to the workspace.
// KG: groups of four waves, each with every KG-th tile of queries.
template <int D, Form FORM, bool SPLIT, int KG>
__global__ __launch_bounds__(kThreads * KG, 2) void attn_dkv_kernel(AttnArgs a, AttnGrads gr, BwdWork w) {
  __shared__ __attribute__((aligned(1024))) DkvLds<D, KG> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wave / kWaves, wv = wave % kWaves;
  const int g = lane >> 5, l32 = lane & 31;
  const int tiles = (int)((a.M + kKeysWg - 1) / kKeysWg), group = a.hq / a.hk;
  int place, hk;
  const int split = SPLIT ? blockIdx.x % w.splits : 0;
  // a split's query heads, and its tiles' number
  const int hstep = SPLIT ? w.heads : 1, hfirst = split & (hstep - 1), tsplits = SPLIT ? w.splits / hstep : 1;
  const int tsplit = split / hstep;
  unit_place(SPLIT ? blockIdx.x / w.splits : blockIdx.x, tiles, a.hk, place, hk);
  const int k0 = place * kKeysWg;                 // under a causal mask: the most seen first
  const int kw = k0 + 32 * wv, key = kw + l32;    // this wave's and this lane's first key
  const bool live = key < a.M;
  const int64_t ldo = (int64_t)a.hq * a.d;
  const int qtiles = (int)((a.M + kRows - 1) / kRows);
  constexpr int kTileBytes = kRows * D * 2;
  const int qt0 = lds_address(&lds.rows[kg][0][0][0]), ot0 = qt0 + 2 * kTileBytes;
  const int stat0 = lds_address(&lds.stat[kg][0][0]), span0 = lds_address(&lds.span[kg][0][0]);

  // the tiles of queries: waves 0 and 1 copy Q, 2 and 3 dO
  Tile<D, false> tile;
  tile.init((uint32_t)(wv < 2 ? a.ldq : ldo) * 2, (uint32_t)a.d * 2, lane, wv & 1);
  auto fetch = [&](int head, int qt, int slot) {
    const int q0 = qt * kRows;
    TileSource s;
    s.init(wv < 2 ? a.Q : gr.dO, wv < 2 ? a.ldq : ldo, head, a.d, a.M);
    s.copy(tile, q0, (wv < 2 ? qt0 : ot0) + slot * kTileBytes, wv & 1);
    // rows past the last: their statistics are there, their spans read as zero, empty
    const int row = lane * 4, at = slot * (kRows * 8);
    if (wv == 0) lload_lds4(lrsrc(w.stat + head * w.ld + q0, kRows * 8), stat0 + at, row);
    if (wv == 2) lload_lds4(lrsrc(a.spans + 2 * (int64_t)q0, a.M > q0 ? (a.M - q0) * 8 : 0), span0 + at, row);
  };
  // The tiles that see any of the workgroup's keys, 64 at a time: bit t of `hits` is tile
  // block + t, or one of the groups' KG tiles from there; `none` see nothing of the wave's
  // keys, in `whole` every query sees them all.
  int block = 0;
  uint64_t hits = 0, none = 0, whole = 0;
  auto scan = [&](int from) {  // the first block of tiles from `from` with a hit
    for (block = from; block < qtiles; block += 64) {
      const int t = block + lane;
      const int4 r = t < qtiles ? w.reach[t] : int4{0x7FFFFFFF, 0, 0x7FFFFFFF, 0};
      hits = __ballot(r.x < k0 + kKeysWg && r.y > k0 && (!SPLIT || (lane / KG & (tsplits - 1)) == tsplit));
      if constexpr (KG == 2) hits = (hits | hits >> 1) & 0x5555555555555555u;
      none = __ballot(r.x >= kw + 32 || r.y <= kw);
      whole = __ballot(r.z <= kw && r.w >= kw + 32);
      if (hits) return;
    }
  };

  const float c = a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e, in2 = a.cap > 0.0f ? 2.0f * c / a.cap : 0.0f;
  Reader<D> read;
  read.init(lane);
  u32x4 kf[D / 16];
  load_rows<D>(kf, a.K + (int64_t)key * a.ldk + (int64_t)hk * a.d, live, a.d, g);
  const int vt = lds_address(&lds.v[0]);
  {
    Tile<D, false> tv;
    tv.init((uint32_t)a.ldv * 2, (uint32_t)a.d * 2, lane, wv);
    TileSource s;
    s.init(a.V, a.ldv, hk, a.d, a.M);
    if (KG == 1 || kg == 0) s.copy(tv, k0, vt, wv);
    if (KG == 1 || kg == 1) s.copy(tv, k0 + 64, vt + 64 * D * 2, wv);
  }
  f32x16 dk[D / 32], dv[D / 32];

  auto step = [&](int head, int q0, int slot, bool masked, auto careful) {
    constexpr bool kCareful = decltype(careful)::value;
    constexpr int kGroups = D / 16, kTiles = D / 32;
    const uint32_t qt = qt0 + slot * kTileBytes, ot = ot0 + slot * kTileBytes;
    const uint32_t qr = qt + read.row, dr = ot + read.row, vr = vt + 32 * wv * D * 2 + read.row;
    f32x16 z[2];  // scores, then p; dP, then dS
    zero(z);
    // Reads run ahead as far as registers go: all of the scores' at once, then dP's pairs in
    // the place of those that the products have taken.
    constexpr int kPairs = kGroups / 2 < 3 ? kGroups / 2 : 3;
    u32x4 f[kGroups];
#pragma unroll
    for (int kk = 0; kk < kGroups; ++kk) f[kk] = row_frag<D>(qr, 0, kk);
#pragma unroll
    for (int kk = 0; kk < kGroups; ++kk) {
      z[0] = lmfma(f[kk], kf[kk], z[0]);
      if (kk < 2 * kPairs) f[kk] = row_frag<D>(kk & 1 ? vr : dr, 0, kk >> 1);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int kk = 0; kk < kGroups; ++kk) {
      const int at = 2 * (kk % kPairs);
      z[1] = lmfma(f[at], f[at + 1], z[1]);
      if (kk + kPairs < kGroups) {
        f[at] = row_frag<D>(dr, 0, kk + kPairs);
        f[at + 1] = row_frag<D>(vr, 0, kk + kPairs);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const f32x4 *stat = reinterpret_cast<const f32x4 *>(lds.stat[kg][slot]);
    const float slope2 = FORM != kPlain && a.slopes ? a.slopes[head] * kLog2e : 0.0f;
    const float away = (float)(key - (q0 + 4 * g));
    if constexpr (FORM == kCapped) tanh_all(reinterpret_cast<f32x16(&)[1]>(z[0]), in2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 s0 = stat[4 * q + 2 * g], s1 = stat[4 * q + 2 * g + 1];
      const float lse2[4] = {s0[0], s0[2], s1[0], s1[2]}, delta[4] = {s0[1], s0[3], s1[1], s1[3]};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int v = 4 * q + e;
        float p, slack = 1.0f;
        if constexpr (FORM != kPlain) {
          const float y = z[0][v] * (FORM == kCapped ? cap2 : c);
          if constexpr (FORM == kCapped) slack = 1.0f - z[0][v] * z[0][v];
          p = __builtin_amdgcn_exp2f(__builtin_fmaf(-slope2, __builtin_fabsf(away - (float)(8 * q + e)), y) - lse2[e]);
        } else {
          p = __builtin_amdgcn_exp2f(__builtin_fmaf(z[0][v], c, -lse2[e]));
        }
        z[0][v] = p;
        z[1][v] = p * (z[1][v] - delta[e]);
        if constexpr (FORM == kCapped) z[1][v] *= slack;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (masked) {
      const int4 *span = reinterpret_cast<const int4 *>(lds.span[kg][slot]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int4 r0 = span[4 * q + 2 * g], r1 = span[4 * q + 2 * g + 1];
        const int lo[4] = {r0.x, r0.z, r1.x, r1.z}, hi[4] = {r0.y, r0.w, r1.y, r1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool seen = key >= lo[e] && key < hi[e];
          z[0][4 * q + e] = seen ? z[0][4 * q + e] : 0.0f;
          z[1][4 * q + e] = seen ? z[1][4 * q + e] : 0.0f;
        }
      }
    }
    const uint32_t qc = qt + read.col, oc = ot + read.col;
    u32x4 p[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) p[b][0] = pack8(z[0], b), p[b][1] = pack8(z[1], b);
    constexpr int kOps = 2 * kTiles, kAhead = 2;
    if constexpr (kCareful) {
#pragma unroll
      for (int i = 0; i < kOps; ++i) {
        const int b = i / kTiles, e = i % kTiles;
        u32x4 o = col_frag<D>(oc, e, b), q = col_frag<D>(qc, e, b);
        if (masked) o = finite(o), q = finite(q);
        dv[e] = lmfma(o, p[b][0], dv[e]);
        dk[e] = lmfma(q, p[b][1], dk[e]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (masked) {
        const int *span = lds.span[kg][slot];
        for (uint64_t odd = odd_rows<D, kRows>(ot, lane); odd; odd &= odd - 1) {
          const int r = (int)__builtin_ctzll(odd);
          spoil<D>(dv, ot, r, key >= span[2 * r] && key < span[2 * r + 1], g);
        }
        for (uint64_t odd = odd_rows<D, kRows>(qt, lane); odd; odd &= odd - 1) {
          const int r = (int)__builtin_ctzll(odd);
          spoil<D>(dk, qt, r, key >= span[2 * r] && key < span[2 * r + 1], g);
        }
      }
      return;
    }
    u32x4 w[kAhead + 1][2];
    auto cols = [&](int n) {
      w[n % (kAhead + 1)][0] = col_frag<D>(oc, n % kTiles, n / kTiles);
      w[n % (kAhead + 1)][1] = col_frag<D>(qc, n % kTiles, n / kTiles);
    };
#pragma unroll
    for (int n = 0; n < kAhead; ++n) cols(n);
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
      if (i + kAhead < kOps) cols(i + kAhead);
      const int b = i / kTiles, e = i % kTiles;
      dv[e] = lmfma(w[i % (kAhead + 1)][0], p[b][0], dv[e]);
      dk[e] = lmfma(w[i % (kAhead + 1)][1], p[b][1], dk[e]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const int past = (hk + 1) * group;
  auto walk = [&](auto careful) {
    zero(dk);
    zero(dv);
    int head = hk * group + hfirst, slot = 0;
    scan(0);
    if (hits) fetch(head, block + (int)__builtin_ctzll(hits) + kg, 0);
    while (hits) {
      const int at = (int)__builtin_ctzll(hits) + kg, q0 = (block + at) * kRows, h = head;
      const bool seen = !(none >> at & 1), masked = !(whole >> at & 1);
      hits &= hits - 1;
      if (!hits) scan(block + 64);
      if (!hits && (head += hstep) < past) scan(0);  // the next head of the group
      tile_sync();
      if (hits) fetch(head, block + (int)__builtin_ctzll(hits) + kg, slot ^ 1);
      if (seen) step(h, q0, slot, masked, careful);
      slot ^= 1;
    }
  };
  walk(std::false_type{});
  // (as in the forward: taken again if what masked queries hold has spoiled a sum)
  if (any_wave(!(all_finite(dk) && all_finite(dv)), lds.spoiled, wave, kWaves * KG)) {
    // (the keys again: kept for this pass, a register of the first one's products was spilled, whose
    // return waits for the copies: 4001 tokens in 9 documents 154 us, so 150)
    load_rows<D>(kf, a.K + (int64_t)key * a.ldk + (int64_t)hk * a.d, live, a.d, g);
    walk(std::true_type{});
  }
  __syncthreads();  // the last tiles are read
  __builtin_amdgcn_s_waitcnt(0);  // no copy may land after the workgroup's end
  if constexpr (KG > 1) {
    static_assert(KG == 2, "one group's sums go to the other");
    join_groups<D>(dk, lds.join[wv], kg, lane);
    join_groups<D>(dv, lds.join[wv], kg, lane);
    if (kg == 1) return;
  }
  const int64_t at = ((int64_t)key * a.hk + hk) * a.d;
  if constexpr (!SPLIT) {
    store_row<D>(gr.dK + at, dk, a.scale, live, a.d, g);
    store_row<D>(gr.dV + at, dv, 1.0f, live, a.d, g);
  } else {
    const int64_t all = a.M * a.hk * a.d;
    store_sums<D>(w.part + split * all + at, dk, live, a.d, g);
    store_sums<D>(w.part + (w.splits + split) * all + at, dv, live, a.d, g);
  }
}

// dK and dV from the splits' sums, eight values a thread, in the splits' order.
__global__ __launch_bounds__(kThreads) void attn_dkv_sum_kernel(const float *part, int splits, int64_t n, float scale,
                                                                 uint16_t *dK, uint16_t *dV) {
  const int64_t i = 8 * ((int64_t)blockIdx.x * kThreads + threadIdx.x);
  const bool second = i >= n;
  const int64_t at = second ? i - n : i;
  if (at >= n) return;
  const float *p = part + (second ? splits * n : 0) + at;
  f32x4 x{0.0f, 0.0f, 0.0f, 0.0f}, y = x;
  for (int s = 0; s < splits; ++s) {
    x += *reinterpret_cast<const f32x4 *>(p + s * n);
    y += *reinterpret_cast<const f32x4 *>(p + s * n + 4);
  }
  const float by = second ? 1.0f : scale;
  const u32x4 o{pack_bf16x2(x[0] * by, x[1] * by), pack_bf16x2(x[2] * by, x[3] * by), pack_bf16x2(y[0] * by, y[1] * by),
                pack_bf16x2(y[2] * by, y[3] * by)};
  *reinterpret_cast<u32x4 *>((second ? dV : dK) + at) = o;
}

size_t attn_bwd_workspace(int64_t M, int64_t hq, int64_t hk, int64_t d) {
  const int64_t ld = padded(M), s = bwd_work(M, hq, hk, nullptr).splits;
  return (size_t)(hq * ld * 8 + ld / 32 * 16 + (s > 1 ? 8 * s * M * hk * d : 0));
}

template <int D, Form FORM>
static hipError_t launch_both(const AttnArgs &a, const AttnGrads &g, const BwdWork &w, hipStream_t st) {
  const dim3 gq((uint32_t)((a.M + kRowsWg - 1) / kRowsWg * a.hq));
  const dim3 gk((uint32_t)((a.M + kKeysWg - 1) / kKeysWg * a.hk * w.splits));
  // Two groups of waves where one leaves compute units half empty; a second round of workgroups
  // (there is room for one of each kind a unit) is short if there are many tokens.  Backward with
  // one and two, 128 values a head (64 take the same rule), causal:
  //   256 workgroups   256 tokens 44, 44 us   1000   83, 81    2048  127, 121   4096  215, 201
  //   288 to 384       1000 tokens 110, 118   1500  106, 101   2000  148, 148   4096  245, 228
  //   512              1000 tokens 97, 105    2048  170, 170   8192  564, 532
  //   768 and more     2048 tokens 213, 228
  const bool two = gq.x <= 256 || (gq.x <= 512 && a.M > 1024);
  const hipError_t e = two ? launch(attn_dq_kernel<D, FORM, 2>, gq, kThreads * 2, st, a, g, w)
                           : launch(attn_dq_kernel<D, FORM, 1>, gq, kThreads, st, a, g, w);
  if (e != hipSuccess) return e;
  void (*dkv)(AttnArgs, AttnGrads, BwdWork) = w.splits > 1   ? attn_dkv_kernel<D, FORM, true, 2>
                                              : w.groups > 1 ? attn_dkv_kernel<D, FORM, false, 2>
                                                             : attn_dkv_kernel<D, FORM, false, 1>;
  return launch(dkv, gk, kThreads * w.groups, st, a, g, w);
}

hipError_t launch_attn_bwd(const AttnArgs &a, const AttnGrads &g, void *ws, hipStream_t st) {
  const BwdWork w = bwd_work(a.M, a.hq, a.hk, ws);
  hipError_t e;
  switch (form_of(a.cap, a.slopes)) {
    case kPlain: e = a.d <= 64 ? launch_both<64, kPlain>(a, g, w, st) : launch_both<128, kPlain>(a, g, w, st); break;
    case kBiased: e = a.d <= 64 ? launch_both<64, kBiased>(a, g, w, st) : launch_both<128, kBiased>(a, g, w, st); break;
    default: e = a.d <= 64 ? launch_both<64, kCapped>(a, g, w, st) : launch_both<128, kCapped>(a, g, w, st);
  }
  if (e != hipSuccess || w.splits == 1) return e;
  const int64_t n = a.M * a.hk * a.d;
  return launch(attn_dkv_sum_kernel, dim3((uint32_t)((2 * n / 8 + kThreads - 1) / kThreads)), kThreads, st, w.part,
                w.splits, n, a.scale, g.dK, g.dV);
}

}  // namespace ql
