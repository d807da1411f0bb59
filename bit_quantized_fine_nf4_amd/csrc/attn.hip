// Attention of packed tokens forward, for gfx950, and the spans of packed documents.
//
// Query i sees the keys lo_i <= j < hi_i of its span:
//   z_ij = scale q_i . k_j,  capped: cap tanh(z / cap),  biased: z - slope |i - j|
//   O_i  = sum_j p_ij v_j with p = softmax over the span,   lse_i = log sum_j exp(z_ij)
// in one pass over the keys with the running maximum and sum; neither z nor p is stored.
//
// A workgroup has 128 queries of a head, a wave 32 of them in its lanes.  Both products are
// formed transposed (z^T = K Q^T, O^T = V^T p^T), so a lane holds one query's scores and
// outputs: the maximum, the sum and the rescaling are a lane's own, the weights go to the
// second product in registers.  64 keys and values at a time go through LDS, two slots of
// each; a tile that some query of the wave does not see wholly takes the masked form.
// The weights are rounded to bf16 for the second product (their sum is not): like the
// operands, by up to 2^-8 of each.
//
// Bound by the matrix cores and the weights' vector operations, which share a SIMD: two
// waves on each take turns, one in its products while the other is in its softmax.
//
// The kernels of 64 values hold 124 to 126 registers, of 128 values 177 to 178 (capped 202 and 254).
// Measured, causal, heads of 128: 8192 tokens of 64 heads for 8 1.04 ms, 1.06 PFLOP/s, matrix
// cores busy 57 % of the cycles (1.14 in twelve traced passes, whose clock falls); 2048 tokens of
// 64 heads 80 to 92 us, 0.86 PFLOP/s (at the former's rate 65: two rounds of workgroups, each
// with a start and an end), busy 39 %; no bank conflicts.  Slower: six waves a workgroup; the
// next tile's products between this one's weights (1.35 ms).
//
// Heads of 72 to 120 values take all products of 128, those of 8 to 56 those of 64: 2048 tokens
// of 64 heads of 64, 80, 96, 112 and 128 values 61, 72, 74, 81 and 80 us.

#include "attn_tiles.h"

namespace ql {
namespace {

constexpr int kQueries = 128;  // per workgroup
constexpr int kKeys = 64;      // per tile

}  // namespace

// KG: groups of four waves, each with every KG-th tile of keys and its own slots.  With two a
// workgroup's queries have twice the waves; their results are joined through LDS.
template <int D, Form FORM, int KG>
__global__ __launch_bounds__(kThreads * KG, 2) void attn_fwd_kernel(AttnArgs a, uint16_t *O, float *lse) {
  __shared__ __attribute__((aligned(1024))) uint16_t ring[KG][4 * kKeys * D];  // K, V; two slots
  __shared__ int ends[2 * kWaves], spoiled[kWaves * KG];
  __shared__ f32x2 stats[kWaves][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = wave / kWaves, wv = wave % kWaves;
  const int g = lane >> 5, l32 = lane & 31;
  const int tiles = (int)((a.M + kQueries - 1) / kQueries);
  int place, head;
  unit_place(blockIdx.x, tiles, a.hq, place, head);
  const int64_t q0 = (int64_t)(tiles - 1 - place) * kQueries;  // under a causal mask: the longest first
  const int64_t row = q0 + 32 * wv + l32;
  const bool live = row < a.M;
  const int hk = head / (a.hq / a.hk);
  const Span span = span_of(a.spans, row, a.M);
  const Reach reach = reach_of(span);
  if (kg == 0 && lane == 0) ends[wv] = reach.lo, ends[kWaves + wv] = reach.hi;
  u32x4 qf[D / 16];
  load_rows<D>(qf, a.Q + row * a.ldq + (int64_t)head * a.d, live, a.d, g);
  __syncthreads();
  int first = ends[0], last = ends[kWaves];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    first = ends[w] < first ? ends[w] : first;
    last = ends[kWaves + w] > last ? ends[kWaves + w] : last;
  }
  first = __builtin_amdgcn_readfirstlane(first < last ? first : last);  // (nothing is seen: first was INT_MAX)
  last = __builtin_amdgcn_readfirstlane(last);

  f32x16 acc[D / 32];
  float top, sum;  // in units of log2; the sum over this lane half's keys
  const float c = a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e, in2 = a.cap > 0.0f ? 2.0f * c / a.cap : 0.0f;
  const float slope2 = FORM != kPlain && a.slopes ? a.slopes[head] * kLog2e : 0.0f;

  constexpr int kTileBytes = kKeys * D * 2;
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

  auto step = [&](int k0, int slot, bool masked, auto careful) {
    constexpr bool kCareful = decltype(careful)::value;
    const uint32_t ks = base + slot * kTileBytes + read.row;
    const uint32_t vs = base + (2 + slot) * kTileBytes + read.col;
    f32x16 z[2];
    zero(z);
    // fragments four groups ahead: all at once would not leave room for the sums
    constexpr int kGroups = D / 16;
    u32x4 kf[3][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) kf[i >> 1][i & 1] = row_frag<D>(ks, i & 1, i >> 1);
#pragma unroll
    for (int kk = 0; kk < kGroups; ++kk) {
      if (kk + 2 < kGroups)
#pragma unroll
        for (int i = 0; i < 2; ++i) kf[(kk + 2) % 3][i] = row_frag<D>(ks, i, kk + 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) z[i] = lmfma(kf[kk % 3][i], qf[kk], z[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the weights' phase first: it is what the wave beside this one, in its products, leaves room for
    __builtin_amdgcn_s_setprio(1);
    if constexpr (FORM == kCapped) tanh_all(z, in2);
    if constexpr (FORM != kPlain) {
      const float away = (float)(k0 + 4 * g - (int)row);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const float x = z[t][v] * (FORM == kCapped ? cap2 : c);
          z[t][v] = __builtin_fmaf(-slope2, __builtin_fabsf(away + (float)(32 * t + acc_row(v, 0))), x);
        }
    }
    if (masked) {
      const int from = span.lo - k0 - 4 * g, width = span.hi - span.lo;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int j = 32 * t + acc_row(v, 0);
          z[t][v] = j < from || j - from >= width ? -__builtin_inff() : z[t][v];
        }
    }
    float mx = -__builtin_inff();
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) mx = fmaxf(mx, z[t][v]);
    mx = both_halves_max(mx);
    if constexpr (FORM == kPlain) mx *= c;
    // The reference follows the maximum only when that is 8 above it: weights stay below
    // 2^8, and most tiles need no rescaling.  (Each query by itself: its results do not
    // depend on its neighbours'.)
    const bool up = mx > top + 8.0f;
    if (__any(up)) {
      const float next = up ? mx : top, by = up ? __builtin_amdgcn_exp2f(top - mx) : 1.0f;
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[t][v] *= by;
      sum *= by;
      top = next;
    }
    const float ref = top == -__builtin_inff() ? 0.0f : top;  // no key yet: every weight is exp2(-inf)
    u32x4 p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        z[t][v] = __builtin_amdgcn_exp2f(FORM != kPlain ? z[t][v] - ref : __builtin_fmaf(z[t][v], c, -ref));
        sum += z[t][v];
      }
      p[2 * t] = pack8(z[t], 0);
      p[2 * t + 1] = pack8(z[t], 1);
    }
    __builtin_amdgcn_s_setprio(0);
    if constexpr (kCareful) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          u32x4 v = col_frag<D>(vs, t, b);
          if (masked) v = finite(v);
          acc[t] = lmfma(v, p[b], acc[t]);
          __builtin_amdgcn_sched_barrier(0);
        }
      if (masked) {
        const uint32_t tile = base + (2 + slot) * kTileBytes;
        for (uint64_t odd = odd_rows<D, kKeys>(tile, lane); odd; odd &= odd - 1) {
          const int r = (int)__builtin_ctzll(odd);
          spoil<D>(acc, tile, r, k0 + r >= span.lo && k0 + r < span.hi, g);
        }
      }
    } else {
      u32x4 vf[2][D / 32];
#pragma unroll
      for (int t = 0; t < D / 32; ++t) vf[0][t] = col_frag<D>(vs, t, 0);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b < 3)
#pragma unroll
          for (int t = 0; t < D / 32; ++t) vf[b + 1 & 1][t] = col_frag<D>(vs, t, b + 1);
#pragma unroll
        for (int t = 0; t < D / 32; ++t) acc[t] = lmfma(vf[b & 1][t], p[b], acc[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  auto walk = [&](auto careful) {
    zero(acc);
    top = -__builtin_inff(), sum = 0.0f;
    int slot = 0;
    if (first + kg * kKeys < last) fetch(first + kg * kKeys, 0);
    for (int at = first; at < last; at += KG * kKeys, slot ^= 1) {
      const int k0 = at + kg * kKeys;
      tile_sync();
      if (k0 + KG * kKeys < last) fetch(k0 + KG * kKeys, slot ^ 1);
      if (k0 >= reach.hi || k0 + kKeys <= reach.lo) continue;  // nothing of this wave's
      step(k0, slot, k0 < reach.all_lo || k0 + kKeys > reach.all_hi, careful);
    }
  };
  // What masked tokens hold must not enter, but a weight of zero times an infinity or a NaN
  // is NaN.  A pass that leaves a sum that is not finite is taken again with zeros in the place
  // of such values in masked tiles, and NaN for the queries that see them: to look for them in
  // every masked tile took a third of such a tile's time.  (A query that sees nothing may hold
  // anything, in its own lanes.)
  walk(std::false_type{});
  if (any_wave(span.lo < span.hi && !all_finite(acc), spoiled, wave, kWaves * KG)) walk(std::true_type{});

  sum = both_halves_sum(sum);
  if constexpr (KG > 1) {
    static_assert(KG == 2, "one group's results go to the other");
    f32x4 *join = reinterpret_cast<f32x4 *>(ring) + wv * (D / 8 * 64) + lane;
    __syncthreads();  // the last tiles are read
    if (kg == 1) {
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          join[64 * (4 * t + q)] = f32x4{acc[t][4 * q], acc[t][4 * q + 1], acc[t][4 * q + 2], acc[t][4 * q + 3]};
      stats[wv][lane] = f32x2{top, sum};
    }
    __syncthreads();
    if (kg == 1) return;
    const f32x2 other = stats[wv][lane];
    const float both = fmaxf(top, other[0]), ref = both == -__builtin_inff() ? 0.0f : both;
    const float by = __builtin_amdgcn_exp2f(top - ref), to = __builtin_amdgcn_exp2f(other[0] - ref);
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 x = join[64 * (4 * t + q)];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][4 * q + i] = __builtin_fmaf(to, x[i], by * acc[t][4 * q + i]);
      }
    sum = __builtin_fmaf(to, other[1], by * sum);
    top = both;
  }
  // (a sum that is not a number is no row without keys: it goes on into O and lse)
  const bool any = span.lo < span.hi && !(sum == 0.0f);
  store_row<D>(O + (row * a.hq + head) * a.d, acc, any ? 1.0f / sum : 0.0f, live, a.d, g);
  if (live && g == 0)
    lse[(int64_t)head * a.M + row] = any ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : -__builtin_inff();
}

// Spans of packed documents: document e has the tokens documents[e] <= i < documents[e + 1],
// its first prefix[e] tokens are seen by all of it.  A token of no document sees nothing.
__global__ __launch_bounds__(kThreads) void attn_spans_kernel(const int32_t *documents, int64_t n,
                                                              const int32_t *prefix, int64_t M, bool causal,
                                                              int64_t window, int32_t *spans) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= M) return;
  int64_t lo = 0, hi = 0;
  if (i >= documents[0] && i < documents[n]) {
    int64_t e = 0, past = n;  // the last document that begins at or before i
    while (past - e > 1) {
      const int64_t mid = (e + past) / 2;
      if (documents[mid] <= i) e = mid;
      else past = mid;
    }
    const int64_t begin = documents[e], end = documents[e + 1];
    lo = begin, hi = end;
    if (window > 0 && lo < i - window + 1) lo = i - window + 1;
    if (window > 0 && hi > i + window) hi = i + window;
    if (causal) {
      const int64_t seen = prefix ? begin + (int64_t)prefix[e] : 0;
      hi = seen > i + 1 ? (seen < end ? seen : end) : i + 1;
    }
  }
  spans[2 * i] = (int32_t)(lo < 0 ? 0 : lo);
  spans[2 * i + 1] = (int32_t)(hi > M ? M : hi);
}

hipError_t launch_attn_spans(const int32_t *documents, int64_t n, const int32_t *prefix, int64_t M, bool causal,
                             int64_t window, int32_t *spans, hipStream_t st) {
  const dim3 grid((uint32_t)((M + kThreads - 1) / kThreads));
  return launch(attn_spans_kernel, grid, kThreads, st, documents, n, prefix, M, causal, window, spans);
}

template <int KG>
static hipError_t launch_fwd(const AttnArgs &a, uint16_t *O, float *lse, hipStream_t st) {
  const dim3 grid((uint32_t)((a.M + kQueries - 1) / kQueries * a.hq));
  void (*kernel)(AttnArgs, uint16_t *, float *);
  switch (form_of(a.cap, a.slopes)) {
    case kPlain: kernel = a.d <= 64 ? attn_fwd_kernel<64, kPlain, KG> : attn_fwd_kernel<128, kPlain, KG>; break;
    case kBiased: kernel = a.d <= 64 ? attn_fwd_kernel<64, kBiased, KG> : attn_fwd_kernel<128, kBiased, KG>; break;
    default: kernel = a.d <= 64 ? attn_fwd_kernel<64, kCapped, KG> : attn_fwd_kernel<128, kCapped, KG>;
  }
  return launch(kernel, grid, kThreads * KG, st, a, O, lse);
}

// Two groups of waves where one would leave compute units, which hold two workgroups of four
// waves, half empty or with one long workgroup each.  Heads of 64 values and fewer take the same
// rule, whose sides were measured at 128.  One and two groups, 128 values a head, causal:
//   256 workgroups   256 tokens 12.2, 12.2 us    1000  25.6, 22.0    4096   77, 59    8192  146, 112
//   512              1000 tokens 30.7, 32.7      2048  51.8, 46.7    8192  178, 140
//   768 and more     2048 tokens 60, 72          4096 (1024 workgroups)  138, 152
hipError_t launch_attn_fwd(const AttnArgs &a, uint16_t *O, float *lse, hipStream_t st) {
  return (a.M + kQueries - 1) / kQueries * a.hq <= 512 ? launch_fwd<2>(a, O, lse, st) : launch_fwd<1>(a, O, lse, st);
}

}  // namespace ql
