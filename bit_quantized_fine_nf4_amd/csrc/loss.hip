// Softmax cross entropy of an output head over a large vocabulary without kept logits.
//
// For hidden states H [M][h], a head W [V][h] and labels, with z = H · W^T:
//   lse = log(sum_v exp z_v),   loss = lse - z[label]
//   G   = (softmax(z) - onehot(label)) * dloss,   dH = G · W,   dW = G^T · H
// z (M x V, gigabytes) is never stored: the forward's product keeps, per tile of the
// vocabulary, each token's maximum and sum of exponentials; the backward computes z
// again, piece by piece of the vocabulary, turns each piece into G in bf16 and multiplies
// it at once.  G is rounded to bf16 because it is a matrix-core operand of the two
// gradient products; their sums are float32.  What is rounded is G without the largest
// |dloss|, which multiplies the sums instead: with the mean's one dloss for all tokens a
// label's entry is then -1 (+ its probability) and rounds to almost nothing, where
// -1 / count would be off by up to 2^-9 in every token alike (dH's error against 64 bits
// 2.6e-3 of its norm, now that of its own rounding, 1.7e-3).
//
// Tokens whose label is outside [0, V) (prompt and padding tokens) carry no loss.  The
// others are first gathered into a compact copy of H, so such tokens cost no products
// and whatever their rows hold (NaN included) reaches nothing.  Their number is known
// on the GPU only: launches are sized for all M tokens and the surplus workgroups leave.
// (The forward of at most 32 tokens, one tile either way, takes H as it is.)
//
// Kernels: loss_select_kernel (one workgroup: the compact list), loss_gather_kernel
// (the copy; zeroes the skipped rows of dH), both as loss_collect_kernel where the tokens
// are few, the products of loss_gemm.hip (few tokens) and loss_wide.hip,
// loss_finish_kernel (lse and loss from the tiles' statistics), loss_dh_kernel (sums
// dH's partials and rounds).  Everything is added in a fixed order: no atomics.

#include "loss.h"

namespace ql {
namespace {

inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

constexpr int kSelThreads = 1024;

// Infinities and NaN (an overflowed loss scale) do not count: they stay with their own
// token's G instead of spoiling the common factor.
QL_DEV float largest(float top, float v) {
  const float a = fabsf(v);
  return a < __builtin_inff() && a > top ? a : top;
}

}  // namespace

// The tokens with a label in [0, V), in order: idx[i], label[i], and with `lse` the
// compact lse and dloss and the largest finite |dloss|.  Tokens without one get loss = lse = 0 (forward).
__global__ __launch_bounds__(kSelThreads) void loss_select_kernel(const int64_t *labels, int64_t M, int64_t V,
                                                                  int *count, int *idx, int *label,
                                                                  const float *lse, const float *dloss,
                                                                  float *c_lse, float *c_dloss, float *c_top,
                                                                  float *out_loss, float *out_lse) {
  __shared__ int sums[2][kSelThreads / 64];
  __shared__ float tops[kSelThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  int buf = 0;
  float top = 0.0f;
  for (int64_t m0 = 0; m0 < M; m0 += 4 * kSelThreads, buf ^= 1) {
    int64_t lab[4];
    int ok[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + 4 * tid + j;
      lab[j] = m < M ? labels[m] : -1;
      ok[j] = lab[j] >= 0 && lab[j] < V;
      mine += ok[j];
    }
    int inc = mine;  // inclusive sum over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d, 64);
      if (lane >= d) inc += o;
    }
    if (lane == 63) sums[buf][wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 64; ++w) {
      const int s = sums[buf][w];
      before += w < wave ? s : 0;
      all += s;
    }
    int at = base + before + inc - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + 4 * tid + j;
      if (ok[j]) {
        idx[at] = (int)m;
        label[at] = (int)lab[j];
        if (lse) {
          c_lse[at] = lse[m];
          c_dloss[at] = dloss[m];
          top = largest(top, dloss[m]);
        }
        ++at;
      } else if (out_loss && m < M) {
        out_loss[m] = 0.0f;
        out_lse[m] = 0.0f;
      }
    }
    base += all;
  }
  if (tid == 0) *count = base;
  if (!lse) return;  // the whole workgroup
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kSelThreads / 64; ++w) top = fmaxf(top, tops[w]);
    *c_top = top;
  }
}

// Row i of the compact copy (blocked) = row idx[i] of H (i < n), zero from n up to the next
// 32; with dH, the rows without a label become zero.  A workgroup takes 32 rows and one of
// `parts` shares of their columns; a wave 64 columns at a time, so that it reads whole
// 128-byte lines of eight rows and writes 512 bytes in a piece (4096 x 8192: 25 us; one row
// per wave wrote 64 bytes at a time: 28; 1536 of 2048 rows: 13.8, and 17).
__global__ __launch_bounds__(256) void loss_gather_kernel(const uint16_t *H, int64_t M, int64_t h, int parts,
                                                          const int *count, const int *idx, uint16_t *Hc,
                                                          const int64_t *labels, int64_t V, uint16_t *dH) {
  const int lane = threadIdx.x & 63;
  const int n = *count, pad = (n + 31) / 32 * 32;
  const int64_t i0 = (int64_t)(blockIdx.x / parts) * 32;
  const int64_t first = (int64_t)(blockIdx.x % parts) * 4 + (threadIdx.x >> 6);
  const int c8 = (lane & 7) * 8;
  if (i0 < pad) {
    const uint16_t *src[4];
    bool live[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + 8 * k + (lane >> 3);
      live[k] = i < n;
      src[k] = H + (int64_t)(live[k] ? idx[i] : 0) * h + c8;
    }
    uint16_t *dst = Hc + i0 * h + (lane >> 3) * 32 + (c8 >> 5) * 1024 + (c8 & 31);
    for (int64_t cp = first; cp < h / 64; cp += 4 * parts) {
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = live[k] ? *reinterpret_cast<const u32x4 *>(src[k] + cp * 64) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k) *reinterpret_cast<u32x4 *>(dst + cp * 2048 + k * 256) = v[k];
    }
  }
  if (!dH) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t m = i0 + 8 * k + (lane >> 3);
    if (m < M && (labels[m] < 0 || labels[m] >= V))
      for (int64_t cp = first; cp < h / 64; cp += 4 * parts)
        *reinterpret_cast<u32x4 *>(dH + m * h + cp * 64 + c8) = u32x4{0, 0, 0, 0};
  }
}

// loss_select_kernel and loss_gather_kernel in one, for at most kCollect tokens: every
// workgroup makes the list for itself (the labels are a few KB) and copies its share of
// the rows; workgroup 0 also stores the list.  At 16 tokens of 4096 values the two took
// 9 us and a wait between launches, this one 4.8 us.
constexpr int kCollect = 1024;
__global__ __launch_bounds__(256) void loss_collect_kernel(const uint16_t *H, const int64_t *labels, int64_t M,
                                                           int64_t h, int64_t V, int *count, int *idx, int *label,
                                                           const float *lse, const float *dloss, float *c_lse,
                                                           float *c_dloss, float *c_top, float *out_loss,
                                                           float *out_lse, uint16_t *Hc, uint16_t *dH) {
  constexpr int kWaves = 4, kPer = kCollect / 256;
  __shared__ int list[kCollect];  // by compact token; -1 for the tokens past the last
  __shared__ int sums[kWaves];
  __shared__ float tops[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool store = blockIdx.x == 0;
  int64_t lab[kPer];
  bool ok[kPer];
  int mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int m = kPer * tid + j;
    lab[j] = m < M ? labels[m] : -1;
    ok[j] = lab[j] >= 0 && lab[j] < V;
    mine += ok[j];
    list[m] = -1;
  }
  int inc = mine;  // inclusive sum over the wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d, 64);
    if (lane >= d) inc += o;
  }
  if (lane == 63) sums[wave] = inc;
  __syncthreads();
  int at = inc - mine, n = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    at += w < wave ? sums[w] : 0;
    n += sums[w];
  }
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int m = kPer * tid + j;
    if (ok[j]) {
      list[at] = m;
      if (store) {
        idx[at] = m;
        label[at] = (int)lab[j];
        if (lse) {
          c_lse[at] = lse[m];
          c_dloss[at] = dloss[m];
          top = largest(top, dloss[m]);
        }
      }
      ++at;
    } else if (store && out_loss && m < M) {
      out_loss[m] = 0.0f;
      out_lse[m] = 0.0f;
    }
  }
  if (store) {
    if (tid == 0) *count = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    if (lane == 0) tops[wave] = top;
  }
  __syncthreads();
  if (store && lse && tid == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, tops[w]);
    *c_top = top;
  }
  const int pad = (n + 31) / 32 * 32;
  const int64_t per = h / 8, rows = dH && M > pad ? M : pad;
  for (int64_t e = (int64_t)blockIdx.x * 256 + tid; e < rows * per; e += (int64_t)gridDim.x * 256) {
    const int i = (int)(e / per);
    const int64_t c = e % per;
    if (i < pad) {
      const int m = list[i];
      u32x4 v{0, 0, 0, 0};
      if (m >= 0) v = *reinterpret_cast<const u32x4 *>(H + m * h + c * 8);
      *reinterpret_cast<u32x4 *>(Hc + (int64_t)(i >> 5) * h * 32 + (i & 31) * 32 + (c >> 2) * 1024 + (c & 3) * 8) = v;
    }
    if (dH && i < M && (labels[i] < 0 || labels[i] >= V))
      *reinterpret_cast<u32x4 *>(dH + i * h + c * 8) = u32x4{0, 0, 0, 0};
  }
}

// lse and loss of token i from the tiles' (max, sum): compact tokens, or with `labels` all
// M, of which those without a label in [0, V) get 0.  One wave per token.
__global__ __launch_bounds__(256) void loss_finish_kernel(const f32x2 *part, int64_t ldp, int tiles, const int *count,
                                                          const int *idx, const int64_t *labels, int64_t M, int64_t V,
                                                          const float *zlab, float *loss, float *lse) {
  constexpr int kAhead = 8;  // tiles in flight per lane
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= (labels ? M : *count)) return;
  const int64_t token = labels ? i : idx[i];
  const bool live = !labels || (labels[i] >= 0 && labels[i] < V);
  const float z = live ? zlab[i] : 0.0f;  // (written for these tokens only)
  float mx = -__builtin_inff(), s = 0.0f;
  for (int t0 = lane; t0 < tiles; t0 += 64 * kAhead) {
    f32x2 a[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      a[k] = t0 + 64 * k < tiles ? part[(int64_t)(t0 + 64 * k) * ldp + i] : f32x2{0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (a[k][1] == 0.0f) continue;  // no rows of the vocabulary
      const float m = fmaxf(mx, a[k][0]);
      s = s * __expf(mx - m) + a[k][1] * __expf(a[k][0] - m);
      mx = m;
    }
  }
  float top = mx;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  s *= mx == -__builtin_inff() ? 0.0f : __expf(mx - top);  // a lane without tiles
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  if (lane == 0) {
    const float l = top + logf(s);
    lse[token] = live ? l : 0.0f;
    loss[token] = live ? l - z : 0.0f;
  }
}

// dH[idx[i]] = bf16(top * sum over the splits of part[split][i]), eight values per thread.
// splits 0: as head_splits chooses for the tokens there are, [splits][n][h]; otherwise
// [splits][M][h].
__global__ __launch_bounds__(256) void loss_dh_kernel(const float *part, int splits, int64_t M, int64_t rows,
                                                      int64_t first, int64_t h, const int *count, const int *idx,
                                                      const float *c_top, uint16_t *dH) {
  const int n = *count;
  if (n == 0) return;
  const float top = *c_top;
  const int64_t stride = (splits ? M : n) * h;
  if (!splits) splits = head_splits(n, h, first, rows);
  const int64_t per = h / 8, total = (int64_t)n * per;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t i = e / per, c = e % per * 8;
    const float *src = part + i * h + c;
    f32x4 a = *reinterpret_cast<const f32x4 *>(src), b = *reinterpret_cast<const f32x4 *>(src + 4);
    int s = 1;
    for (; s + 7 < splits; s += 8) {  // eight splits' loads in flight, added in order
      f32x4 u[8], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float *q = src + (int64_t)(s + k) * stride;
        u[k] = *reinterpret_cast<const f32x4 *>(q);
        w[k] = *reinterpret_cast<const f32x4 *>(q + 4);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        a += u[k];
        b += w[k];
      }
    }
    for (; s < splits; ++s) {
      const float *q = src + (int64_t)s * stride;
      a += *reinterpret_cast<const f32x4 *>(q);
      b += *reinterpret_cast<const f32x4 *>(q + 4);
    }
    a *= top;
    b *= top;
    *reinterpret_cast<u32x4 *>(dH + (int64_t)idx[i] * h + c) =
        u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
  }
}

namespace {

// The backward's pieces of the vocabulary: G's piece [M][piece] stays near 256 MB, what
// the last-level cache holds, so the products that follow read it from there.
int64_t loss_piece(int64_t M, int64_t V) {
  int64_t p = ((int64_t)1 << 27) / M / 256 * 256;
  p = p < 4096 ? 4096 : (p > (1 << 20) ? 1 << 20 : p);
  const int64_t all = cdiv(V, 256) * 256;
  return p < all ? p : all;
}

// At most 64 tokens: splits of dH's sum over the vocabulary until about 512 workgroups
// read the head, each at least 512 entries of it.
int few_splits(int64_t h, int64_t piece) {
  int64_t s = cdiv(512, cdiv(h, 256));
  s = s > piece / 512 ? piece / 512 : s;
  return (int)(s < 1 ? 1 : s);
}

// Rows of partial sums: every token once, and room to split the sums of up to 8192.
int64_t partial_rows(int64_t M) { return M > 8192 ? M : (16 * M < 8192 ? 16 * M : 8192); }

struct LossLayout {
  size_t count, top, idx, label, lse, dloss, hc, stat, zlab, g, part, total;
  int64_t piece, kper, rows;  // kper and splits: at most 64 tokens
  int splits;
};

LossLayout loss_layout(int64_t M, int64_t h, int64_t V, bool bwd) {
  LossLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += (bytes + 255) / 256 * 256; return at; };
  L.count = take(4);
  L.top = take(4);
  L.idx = take((size_t)M * 4);
  L.label = take((size_t)M * 4);
  // The compact copy's rows: whole blocks (readers stop there); none where the forward takes
  // H as it is.
  L.hc = take(!bwd && M <= kFewTokens ? 0 : (size_t)(cdiv(M, 32) * 32) * h * 2);
  if (!bwd) {
    L.stat = take((size_t)logit_parts(M, h, V) * M * 8);
    L.zlab = take((size_t)M * 4);
  } else {
    L.lse = take((size_t)M * 4);
    L.dloss = take((size_t)M * 4);
    L.piece = loss_piece(M, V);
    // G's rows: whole tiles of the kernel that writes them (a row more than M costs 2 bytes a
    // word: one token of 2^20 words takes 64 MB)
    const int64_t tile = M <= kFewTokens ? kFewTokens : M <= 128 ? 128 : 256;
    L.g = take((size_t)(cdiv(M, tile) * tile) * L.piece * 2);
    L.rows = partial_rows(M);
    if (M <= 64) {
      L.kper = cdiv(cdiv(L.piece, few_splits(h, L.piece)), 64) * 64;
      L.splits = (int)cdiv(V < L.piece ? V : L.piece, L.kper);  // those that the first piece fills
      L.rows = (int64_t)L.splits * M;
    }
    L.part = take((size_t)L.rows * h * 4);
  }
  L.total = off;
  return L;
}

template <typename T>
T *at(void *ws, size_t off) { return reinterpret_cast<T *>(reinterpret_cast<char *>(ws) + off); }

// The compact tokens: list, their lse and dloss (backward), the copy of their rows.
struct Compact {
  int *count, *idx, *label;
  float *lse, *dloss, *top;
  uint16_t *H;
};

hipError_t collect(const LossArgs &a, const Compact &c, const float *lse, const float *dloss, float *out_loss,
                   float *out_lse, uint16_t *dH, hipStream_t st) {
  if (a.M <= kCollect) {
    const int64_t groups = cdiv(cdiv(a.M, 32) * 32 * (a.h / 8), 256);
    return launch(loss_collect_kernel, (unsigned)(groups < 1024 ? groups : 1024), 256, st, a.H, a.labels, a.M, a.h,
                  a.V, c.count, c.idx, c.label, lse, dloss, c.lse, c.dloss, c.top, out_loss, out_lse, c.H, dH);
  }
  hipError_t e = launch(loss_select_kernel, 1, kSelThreads, st, a.labels, a.M, a.V, c.count, c.idx, c.label, lse,
                        dloss, c.lse, c.dloss, c.top, out_loss, out_lse);
  if (e != hipSuccess) return e;
  const int parts = (int)cdiv(a.h / 64, 16);  // four columns' turns per wave
  return launch(loss_gather_kernel, (unsigned)(cdiv(a.M, 32) * parts), 256, st, a.H, a.M, a.h, parts,
                (const int *)c.count, (const int *)c.idx, c.H, a.labels, a.V, dH);
}

}  // namespace

bool loss_supported(int64_t M, int64_t h, int64_t V) {
  // 32-bit offsets of 256 rows of the head, 32-bit tile numbers and thread counts
  return h <= ((int64_t)1 << 20) && V <= ((int64_t)1 << 24) && M <= ((int64_t)1 << 24) &&
         cdiv(M, 256) * cdiv(V, 128) < ((int64_t)1 << 24);
}

size_t loss_fwd_workspace(int64_t M, int64_t h, int64_t V) { return loss_layout(M, h, V, false).total; }
size_t loss_bwd_workspace(int64_t M, int64_t h, int64_t V) { return loss_layout(M, h, V, true).total; }

hipError_t launch_loss_fwd(const LossArgs &a, float *loss, float *lse, void *ws, hipStream_t st) {
  const LossLayout L = loss_layout(a.M, a.h, a.V, false);
  int *count = at<int>(ws, L.count), *idx = at<int>(ws, L.idx), *label = at<int>(ws, L.label);
  uint16_t *Hc = at<uint16_t>(ws, L.hc);
  LogitParams p{};
  p.W = a.W, p.H = Hc, p.count = count, p.label = label, p.h = a.h, p.v0 = 0, p.nvoc = a.V;
  p.part = at<f32x2>(ws, L.stat), p.ldp = a.M, p.zlab = at<float>(ws, L.zlab);
  hipError_t e;
  if (a.M <= kFewTokens) {
    p.H = a.H, p.labels = a.labels, p.M = a.M;
    e = launch_logit_stats_few(p, st);
  } else {
    e = collect(a, Compact{count, idx, label, nullptr, nullptr, nullptr, Hc}, nullptr, nullptr, loss, lse, nullptr, st);
    if (e != hipSuccess) return e;
    e = launch_logit_stats(p, a.M, st);
  }
  if (e != hipSuccess) return e;
  return launch(loss_finish_kernel, (unsigned)cdiv(a.M, 4), 256, st, (const f32x2 *)p.part, p.ldp,
                logit_parts(a.M, a.h, a.V), (const int *)count, (const int *)idx, p.labels, a.M, a.V,
                (const float *)p.zlab, loss, lse);
}

hipError_t launch_loss_bwd(const LossArgs &a, const float *lse, const float *dloss, uint16_t *dH, uint16_t *dW,
                           void *ws, hipStream_t st) {
  const LossLayout L = loss_layout(a.M, a.h, a.V, true);
  int *count = at<int>(ws, L.count), *idx = at<int>(ws, L.idx), *label = at<int>(ws, L.label);
  uint16_t *Hc = at<uint16_t>(ws, L.hc);
  float *c_lse = at<float>(ws, L.lse), *c_dl = at<float>(ws, L.dloss), *top = at<float>(ws, L.top);
  hipError_t e = collect(a, Compact{count, idx, label, c_lse, c_dl, top, Hc}, lse, dloss, nullptr, nullptr, dH, st);
  if (e != hipSuccess) return e;
  float *part = at<float>(ws, L.part);
  for (int64_t v0 = 0; v0 < a.V; v0 += L.piece) {
    const int64_t nvoc = a.V - v0 < L.piece ? a.V - v0 : L.piece;
    LogitParams p{};
    p.W = a.W + v0 * a.h, p.H = Hc, p.count = count, p.label = label, p.h = a.h, p.v0 = v0, p.nvoc = nvoc;
    p.lse = c_lse, p.dloss = c_dl, p.top = top, p.G = at<uint16_t>(ws, L.g), p.gblocks = L.piece / 32;
    e = launch_logit_grad(p, a.M, st);
    if (e != hipSuccess) return e;
    HeadGradParams q{};
    q.G = p.G, q.gblocks = L.piece / 32, q.W = p.W, q.H = Hc, q.count = count, q.top = top, q.h = a.h, q.nvoc = nvoc;
    q.kper = L.kper, q.part = part, q.rows = a.M <= 64 ? a.M : L.rows, q.add = v0 > 0;
    q.first = a.V < L.piece ? a.V : L.piece;
    // (at most 64 tokens: the last piece may fill fewer splits; the others' sums are whole)
    e = launch_head_dh(q, a.M, st);
    if (e != hipSuccess) return e;
    if (dW) {
      q.dW = dW + v0 * a.h;
      e = launch_head_dw(q, st);
      if (e != hipSuccess) return e;
    }
  }
  const int64_t groups = cdiv(a.M * (a.h / 8), 256);
  return launch(loss_dh_kernel, (unsigned)(groups < 8192 ? groups : 8192), 256, st, (const float *)part, L.splits, a.M,
                L.rows, a.V < L.piece ? a.V : L.piece, a.h, (const int *)count, (const int *)idx, (const float *)top, dH);
}

}  // namespace ql
