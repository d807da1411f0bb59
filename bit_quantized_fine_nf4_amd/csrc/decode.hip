// Attention of one new token per sequence over a paged key-value cache, for gfx950.
//
// For sequence b with n = lens[b] tokens in the cache, its own key the last of them:
//   z_j = scale q . k_j,  capped: cap tanh(z / cap),  biased: z - slope (n - 1 - j)
//   O   = sum_j softmax(z)_j v_j   over max(0, n - window) <= j < n.
// Bound by reading the keys and values once.  Measured: 48 sequences of up to 8192 tokens, 64
// heads for 8 (152 MB) 32 us and 4 for the join, 4.7 TB/s of the first (with a cap or a bias the
// same within a microsecond, with a window of 1000 tokens 21 us in all); such of 805 MB in all
// 164 us, 4.9 TB/s; one of 2049 tokens, 32 heads (34 MB) 9 and 4 us, too short to fill the
// memory with copies.
//
// An item of work is a stretch of one sequence for up to 16 query heads that share a key
// head.  Lengths are known on the device only: every workgroup sums them and takes the
// stretch that leaves at most 512 items besides the sequences' ends, as many as workgroups fit,
// whatever the lengths, and from its number finds its items.  (A grid by the room for
// tokens spent more on workgroups without work, 6 ns each, than on the others.  With 544 items
// for 512 workgroups one sequence of 2049 tokens took 14.1 us, join included, with 288 12.4.)
// Items of more than 1024 tokens are halved: the ends, which are shorter, then even out (16
// sequences of up to 16000 tokens 122 -> 102 us; those of up to 4000, not halved, 34).  Four
// waves take tiles of 32 tokens in turn, each with its own maximum, sum and outputs and its own
// tile in LDS, so that nothing waits for another wave before the end.  A tile's keys make
// room for the next one's as soon as the scores are formed, its values when the outputs are: a
// wave always has copies in flight.  The heads are the 16 columns of
// v_mfma_f32_16x16x32_bf16: with one head fifteen of them are idle, and the matrix cores still
// take a tenth of the time that the copies take.  The waves' results are joined through
// LDS; those of several stretches through the workspace, in a second kernel.  More than 16 heads
// for a key head are several items, which read its keys and values again, from the last-level
// cache at best: that batch with one key head for 64 heads (20 MB) 30 us, for 16 21.
//
// A copy's rows are of one page (pages have 8 tokens or more): its descriptor begins at the
// row in the page and ends where the sequence does, so rows past the end, like those of a
// page that is not in the cache, read as zero and are masked.

#include "attn_tiles.h"
#include "cache.h"

namespace ql {
namespace {

constexpr int kHeads = 16;     // columns
constexpr int kStep = 32;      // tokens of a wave's tile
constexpr int kMinStretch = kWaves * kStep;
constexpr int kItems = 512;  // items aimed at, and workgroups
constexpr int kLong = 1024;  // tokens: items of more are halved

QL_DEV f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}
// over the four 16-lane groups
QL_DEV float groups_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return both_halves_max(fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])));
}
QL_DEV float groups_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return both_halves_sum(__builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]));
}

template <int D>
struct DecodeLds {
  static constexpr int kTileElems = kStep * D;
  union {
    uint16_t ring[kWaves][2][kTileElems];  // a wave's keys and values
    float out[kWaves][kHeads][D + 4];      // the waves' outputs (rows 4 banks apart)
  };
  float top[kWaves][kHeads], sum[kWaves][kHeads];
};

// Partial results: rows of d outputs, their maximum and sum, and room up to 16 bytes.
__host__ __device__ constexpr int part_width(int d) { return d + 4; }
__host__ __device__ constexpr int rows_per_item(int group) { return group < kHeads ? group : kHeads; }

// The workspace: of each sequence its first stretch in the list of all and how many it has, which
// whoever works on that first one leaves for the join, then the partial results.  (A join whose
// rows looked for them themselves read all lengths for each row: 8192 sequences of 16 heads and
// one token 1.23 ms, now 0.13; 65536 of them 67 and 1.1, where what is left is that every
// workgroup reads all lengths once.)
struct DecodeWork {
  int2 *place;  // [B]
  float *part;
};
__host__ __device__ inline DecodeWork decode_work(int64_t B, void *ws) {
  int2 *place = reinterpret_cast<int2 *>(ws);
  return DecodeWork{place, reinterpret_cast<float *>(place + (B + 31) / 32 * 32)};
}

// The tokens that a sequence sees: [from, n), from the tile of the first on.
struct Seen {
  int n, from, first;
};
QL_DEV Seen seen_of(const DecodeArgs &a, int64_t b) {
  const int64_t room = a.width * a.c.page, given = b < a.B ? a.lens[b] : 0;
  const int n = (int)(given < 0 ? 0 : given > room ? room : given);
  const int from = a.window > 0 && n > a.window ? n - a.window : 0;
  return Seen{n, from, from / kStep * kStep};
}
// Over the 64 lanes: rotations within 16, then the other 16 and the other 32; and the sums of
// the lanes up to each one.
QL_DEV uint32_t lanes_sum(uint32_t x) {
  auto turn = [](uint32_t v, auto by) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + decltype(by)::value, 0xF, 0xF, false);
  };
  x += turn(x, std::integral_constant<int, 1>{});
  x += turn(x, std::integral_constant<int, 2>{});
  x += turn(x, std::integral_constant<int, 4>{});
  x += turn(x, std::integral_constant<int, 8>{});
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = r[0] + r[1];
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(q[0] + q[1]));
}
QL_DEV uint32_t lanes_upto(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false);  // row_shr:1
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);  // row_bcast:15
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);  // row_bcast:31
  return x;
}
QL_DEV int stretches(const Seen &s, int stretch) {  // an empty sequence has one, which writes its zeros
  const int n = s.n - s.first;
  return n > stretch ? (n - 1) / stretch + 1 : 1;
}
// The list of all sequences' stretches, 64 sequences (one a lane) at a time: those from
// `block` on, with `before` stretches before them.
struct Places {
  int stretch;  // tokens, the same in every workgroup
  int block;
  int64_t before;
  Seen seen;        // this lane's sequence,
  int count, upto;  // its stretches, and those of the block up to and with it
  QL_DEV void count_block(const DecodeArgs &a, int lane) {
    count = (int64_t)block + lane < a.B ? stretches(seen, stretch) : 0;
    upto = (int)lanes_upto((uint32_t)count);
  }
  QL_DEV void init(const DecodeArgs &a, int units, int lane) {
    seen = seen_of(a, lane);
    int64_t tiles = 0;  // (a sequence has at most 2^25)
    for (int64_t b = 0; b < a.B; b += 64) {
      const Seen s = b ? seen_of(a, b + lane) : seen;
      tiles += lanes_sum((uint32_t)((s.n - s.first + kStep - 1) / kStep));
    }
    const int64_t whole = tiles * kStep * units, goal = whole > (int64_t)kItems * kLong ? 2 * kItems : kItems;
    const int64_t t = ((whole + goal - 1) / goal + kMinStretch - 1) / kMinStretch * kMinStretch, most = 1 << 30;
    stretch = (int)(t < kMinStretch ? kMinStretch : t < most ? t : most);
    block = 0;
    before = 0;
    count_block(a, lane);
  }
  QL_DEV int all() const { return __builtin_amdgcn_readlane(upto, 63); }
  QL_DEV void next(const DecodeArgs &a, int lane) {
    before += all();
    block += 64;
    seen = seen_of(a, (int64_t)block + lane);
    count_block(a, lane);
  }
};

}  // namespace

template <int D, Form FORM>
__global__ __launch_bounds__(kThreads) void decode_attn_kernel(DecodeArgs a, int hgroups) {
  __shared__ __attribute__((aligned(1024))) DecodeLds<D> lds;
  constexpr int CH = D / 8, kRows = 64 / CH, kCopies = kStep / kRows;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g4 = lane >> 4, l16 = lane & 15;
  const int group = a.hq / a.c.hk, d = a.c.d, page = a.c.page, shift = __builtin_ctz(page);
  const int units = a.c.hk * hgroups;
  // this lane's place in a copy of kRows of the 8 rows from a multiple of 8: the chunk's
  // swizzle goes by the row in the tile, so copies 16 rows apart are alike
  constexpr int kPeriod = 16 / kRows;
  int voff[kPeriod];
#pragma unroll
  for (int i = 0; i < kPeriod; ++i) {
    const int r = kRows * i + lane / CH, e = ((lane % CH) ^ fold<D>(r)) * 8;
    voff[i] = e < d ? ((r & 7) * d + e) * 2 : kOutside;
  }
  const int kbase = lds_address(&lds.ring[wv][0][0]), vbase = lds_address(&lds.ring[wv][1][0]);
  const int64_t page_rows = (int64_t)a.c.hk << shift;
  const float c = a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e, in2 = a.cap > 0.0f ? 2.0f * c / a.cap : 0.0f;

  Places places;
  places.init(a, units, lane);
  const int stretch = places.stretch;
  const DecodeWork work = decode_work(a.B, a.workspace);
  const bool joined = a.width * page > kMinStretch;  // (otherwise there is neither a workspace nor a join)
  for (int64_t item = blockIdx.x;; item += kItems) {
    // (sequence, stretch) number item / units of the list
    const int64_t want = item / units;
    const int unit = (int)(item - want * units);
    while (places.block < a.B && want >= places.before + places.all()) places.next(a, lane);
    if (places.block >= a.B) break;
    const int in_block = (int)(want - places.before);
    const int at = __builtin_amdgcn_readfirstlane((int)__builtin_ctzll(__ballot(places.upto > in_block)));
    const int64_t b = __builtin_amdgcn_readfirstlane(places.block + at);
    const int count = __builtin_amdgcn_readlane(places.count, at);
    const int split = in_block - (__builtin_amdgcn_readlane(places.upto, at) - count);
    if (joined && split == 0 && unit == 0 && threadIdx.x == 0) work.place[b] = int2{(int)want, count};
    const int hk = unit / hgroups, hg = unit - hk * hgroups;
    const int in_group = hg * kHeads + l16;              // this lane's query head in the group
    const bool live = in_group < group;
    const int head = hk * group + (live ? in_group : 0);
    const int n = __builtin_amdgcn_readlane(places.seen.n, at), from = __builtin_amdgcn_readlane(places.seen.from, at);
    const int begin = __builtin_amdgcn_readlane(places.seen.first, at) + split * stretch;
    const int end = n - begin > stretch ? begin + stretch : n;

    u32x4 qf[D / 32];
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      const int e = 32 * kk + 8 * g4;
      qf[kk] = live && e < d ? *reinterpret_cast<const u32x4 *>(a.Q + (b * a.hq + head) * d + e) : u32x4{0, 0, 0, 0};
    }
    f32x4 acc[D / 16];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float top = -__builtin_inff(), sum = 0.0f;
    const float slope2 = FORM != kPlain && a.slopes ? a.slopes[head] * kLog2e : 0.0f;

    // The table is read through the scalar cache: a vector load would be waited for together
    // with the copies in flight.
    typedef const __attribute__((address_space(4))) int32_t TableEntry;
    TableEntry *table = (TableEntry *)(uintptr_t)(a.table + b * a.width);
    // Where the 8 tokens from each multiple of 8 of a tile lie (pages have 8 or more): offset
    // of the first one seen, bytes up to the last, and how many bytes of rows before the
    // window: their offsets, below the descriptor's start, wrap past its end.
    struct Eight {
      int64_t at;
      int bytes, skip;
    } eight[kStep / 8];
    // which of the tile's 32 tokens have a page in the cache
    auto find = [&](int j0) {
      uint32_t paged = 0;
      int p[kStep / 8];
#pragma unroll
      for (int i = 0; i < kStep / 8; ++i) p[i] = table[(j0 + 8 * i < n ? j0 + 8 * i : n - 1) >> shift];
#pragma unroll
      for (int i = 0; i < kStep / 8; ++i) {
        const int j = j0 + 8 * i, skip = from > j ? from - j : 0, left = n - j < 8 ? n - j : 8;
        const bool good = p[i] >= 0 && p[i] < a.c.pages;
        if (good) paged |= 0xFFu << (8 * i);
        const int64_t row = (good ? p[i] : 0) * page_rows + (hk << shift) + (j & (page - 1)) + skip;
        eight[i] = Eight{row * d * 2, good && left > skip ? (left - skip) * d * 2 : 0, skip * d * 2};
      }
      return paged;
    };
    auto fetch = [&](const uint16_t *pages, int at) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const Eight &x = eight[i * kRows / 8];
        lload_lds<false, true>(lrsrc(reinterpret_cast<const char *>(pages) + x.at, x.bytes), at + i * 1024,
                  voff[i % kPeriod] - x.skip, 0);
      }
    };
    // waits until all but the last `kCopies` of this wave's copies have landed, or all
    auto landed = [&](bool more) {
      if (more) __builtin_amdgcn_s_waitcnt((kCopies & 15) | (7 << 4) | ((kCopies >> 4) << 14));
      else __builtin_amdgcn_s_waitcnt(7 << 4);
      asm volatile("" ::: "memory");
    };
    auto reads_done = [&]() {
      __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
      asm volatile("" ::: "memory");
    };
    const uint16_t *ks = lds.ring[wv][0], *vs = lds.ring[wv][1];
    int j0 = begin + wv * kStep;
    uint32_t paged = 0;
    if (j0 < end) {
      paged = find(j0);
      fetch(a.c.k, kbase);
      fetch(a.c.v, vbase);
    }
    for (; j0 < end; j0 += kWaves * kStep) {
      const int following = j0 + kWaves * kStep;
      landed(true);  // the keys
      f32x4 z[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        z[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          const u32x4 k = *reinterpret_cast<const u32x4 *>(ks + (16 * t + l16) * D + (((4 * kk + g4) ^ fold<D>(l16)) << 3));
          z[t] = mfma16(k, qf[kk], z[t]);
        }
      }
      reads_done();
      uint32_t bits = paged;  // the tokens of the tile that count
      if (following < end) {
        paged = find(following);
        fetch(a.c.k, kbase);
      }
      if (j0 < from) bits &= ~0u << (from - j0);
      if (end - j0 < kStep) bits &= (1u << (end - j0)) - 1;
      if constexpr (FORM == kCapped) tanh_all(z, in2);
      float mx = -__builtin_inff();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int at = 16 * t + 4 * g4 + v;
          float x = z[t][v] * (FORM == kCapped ? cap2 : c);
          if constexpr (FORM != kPlain) x = __builtin_fmaf(-slope2, (float)(n - 1 - (j0 + at)), x);
          x = bits >> at & 1 ? x : -__builtin_inff();
          z[t][v] = x;
          mx = fmaxf(mx, x);
        }
      mx = groups_max(mx);
      const float next = fmaxf(top, mx), ref = next == -__builtin_inff() ? 0.0f : next;
      const float by = __builtin_amdgcn_exp2f(top - ref);
      top = next;
      sum *= by;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          z[t][v] = __builtin_amdgcn_exp2f(z[t][v] - ref);
          sum += z[t][v];
        }
      const u32x4 p{pack_bf16x2(z[0][0], z[0][1]), pack_bf16x2(z[0][2], z[0][3]), pack_bf16x2(z[1][0], z[1][1]),
                    pack_bf16x2(z[1][2], z[1][3])};
      landed(following < end);  // the values
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        const int r = 4 * g4 + (l16 >> 2), chunk = 2 * t + ((l16 & 3) >> 1);
        const uint16_t *at = vs + r * D + ((chunk ^ fold<D>(r)) << 3) + 4 * (l16 & 1);
        const u32x4 v = ltr_pair(at, at + 16 * D);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] *= by;
        acc[t] = mfma16(v, p, acc[t]);
      }
      reads_done();
      if (following < end) fetch(a.c.v, vbase);
    }
    sum = groups_sum(sum);
    __syncthreads();  // every wave's tiles are read: the ring gives way to the outputs
    if (g4 == 0) lds.top[wv][l16] = top, lds.sum[wv][l16] = sum;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) *reinterpret_cast<f32x4 *>(&lds.out[wv][l16][16 * t + 4 * g4]) = acc[t];
    __syncthreads();
    const int rows = group - hg * kHeads < kHeads ? group - hg * kHeads : kHeads;
    for (int i = threadIdx.x; i < rows * (d / 4); i += kThreads) {
      const int h = i / (d / 4), e = 4 * (i % (d / 4));
      float best = lds.top[0][h];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) best = fmaxf(best, lds.top[v][h]);
      const float ref = best == -__builtin_inff() ? 0.0f : best;
      float total = 0.0f;
      f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const float by = __builtin_amdgcn_exp2f(lds.top[v][h] - ref);
        total = __builtin_fmaf(by, lds.sum[v][h], total);
        const f32x4 x = *reinterpret_cast<const f32x4 *>(&lds.out[v][h][e]);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(by, x[k], o[k]);
      }
      if (count == 1) {
        const float by = total > 0.0f ? 1.0f / total : 0.0f;
        const u32x2 w{pack_bf16x2(o[0] * by, o[1] * by), pack_bf16x2(o[2] * by, o[3] * by)};
        *reinterpret_cast<u32x2 *>(a.O + (b * a.hq + hk * group + hg * kHeads + h) * d + e) = w;
      } else {
        const int64_t row = item * rows_per_item(group) + h;
        *reinterpret_cast<f32x4 *>(work.part + row * part_width(d) + e) = o;
        if (e == 0) *reinterpret_cast<f32x2 *>(work.part + row * part_width(d) + d) = f32x2{best, total};
      }
    }
    __syncthreads();  // the outputs are read: the ring may be written
  }
}

// The outputs of a row's (sequence, head) stretches weighted by their sums, by PER waves, each
// with every PER-th stretch.  Bound by its launch and the start of its workgroups: four
// waves where there are few rows, with many stretches each (64 rows of 64: 7.1 us, by one wave
// 13.8), one where there are many (48 sequences of 64 heads: 4.9 us, by four 7.9; 512 rows 4.7 and 4.9).
template <int PER>
__global__ __launch_bounds__(kThreads) void decode_join_kernel(DecodeArgs a, int hgroups) {
  __shared__ f32x2 out[kWaves][64];
  __shared__ f32x2 stat[kWaves];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), d = a.c.d;
  const int64_t row = (int64_t)blockIdx.x * (kWaves / PER) + wv / PER, b = row / a.hq;
  if (b >= a.B) return;
  const int group = a.hq / a.c.hk, units = a.c.hk * hgroups, head = (int)(row - b * a.hq);
  const int hk = head / group, in_group = head - hk * group, unit = hk * hgroups + in_group / kHeads;
  const DecodeWork work = decode_work(a.B, a.workspace);
  const int first = work.place[b].x, count = work.place[b].y;
  if (count == 1) return;
  const int64_t step = (int64_t)units * rows_per_item(group) * part_width(d);
  const float *part = work.part + (((int64_t)first * units + unit) * rows_per_item(group) + in_group % kHeads) * part_width(d);
  const int e = 2 * lane < d ? 2 * lane : 0;
  float best = -__builtin_inff(), total = 0.0f, o0 = 0.0f, o1 = 0.0f;
  for (int s0 = wv % PER; s0 < count; s0 += 4 * PER) {
    f32x2 st[4], x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + i * PER;
      const float *p = part + (s < count ? s : s0) * step;
      st[i] = *reinterpret_cast<const f32x2 *>(p + d);
      x[i] = *reinterpret_cast<const f32x2 *>(p + e);
      if (s >= count) st[i] = f32x2{-__builtin_inff(), 0.0f};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float next = fmaxf(best, st[i][0]), ref = next == -__builtin_inff() ? 0.0f : next;
      const float keep = __builtin_amdgcn_exp2f(best - ref), by = __builtin_amdgcn_exp2f(st[i][0] - ref);
      best = next;
      total = __builtin_fmaf(by, st[i][1], total * keep);
      o0 = __builtin_fmaf(by, x[i][0], o0 * keep);
      o1 = __builtin_fmaf(by, x[i][1], o1 * keep);
    }
  }
  if constexpr (PER > 1) {
    static_assert(PER == kWaves, "a workgroup's waves join one row");
    out[wv][lane] = f32x2{o0, o1};
    if (lane == 0) stat[wv] = f32x2{best, total};
    __syncthreads();
    if (wv > 0) return;
    float top = stat[0][0];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) top = fmaxf(top, stat[v][0]);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    total = o0 = o1 = 0.0f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      const float by = __builtin_amdgcn_exp2f(stat[v][0] - ref);
      total = __builtin_fmaf(by, stat[v][1], total);
      o0 = __builtin_fmaf(by, out[v][lane][0], o0);
      o1 = __builtin_fmaf(by, out[v][lane][1], o1);
    }
  }
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
  if (2 * lane < d) *reinterpret_cast<uint32_t *>(a.O + row * d + 2 * lane) = pack_bf16x2(o0 * inv, o1 * inv);
}

// Items: about kItems by the tokens, and a part of one for each sequence and head group.
size_t decode_workspace(int64_t B, int hq, int hk, int64_t capacity) {
  if (capacity <= kMinStretch) return 0;  // one stretch a sequence
  const int64_t group = hq / hk, units = hk * ((group + kHeads - 1) / kHeads);
  // a stretch is at least the tokens' share of an item: whole ones are no more than aimed at
  const int64_t items = 2 * kItems + B * units;
  return (size_t)((B + 31) / 32 * 32 * 8 + items * rows_per_item((int)group) * part_width(kMaxHeadWidth) * 4);
}

hipError_t launch_decode_attn(const DecodeArgs &a, hipStream_t st) {
  const int hgroups = (a.hq / a.c.hk + kHeads - 1) / kHeads;
  const int64_t units = a.c.hk * hgroups, most = (a.width * a.c.page + kMinStretch - 1) / kMinStretch * a.B * units;
  const dim3 grid((uint32_t)(most < kItems ? most : kItems));
  void (*kernel)(DecodeArgs, int);
  switch (form_of(a.cap, a.slopes)) {
    case kPlain: kernel = a.c.d <= 64 ? decode_attn_kernel<64, kPlain> : decode_attn_kernel<128, kPlain>; break;
    case kBiased: kernel = a.c.d <= 64 ? decode_attn_kernel<64, kBiased> : decode_attn_kernel<128, kBiased>; break;
    default: kernel = a.c.d <= 64 ? decode_attn_kernel<64, kCapped> : decode_attn_kernel<128, kCapped>;
  }
  const hipError_t e = launch(kernel, grid, kThreads, st, a, hgroups);
  if (e != hipSuccess || a.width * a.c.page <= kMinStretch) return e;
  const int64_t rows = a.B * a.hq;
  return rows < 512 ? launch(decode_join_kernel<kWaves>, dim3((uint32_t)rows), kThreads, st, a, hgroups)
                      : launch(decode_join_kernel<1>, dim3((uint32_t)((rows + kWaves - 1) / kWaves)), kThreads, st, a,
                               hgroups);
}

}  // namespace ql
