// Residual update with RMS norms before and after a transformer block, for gfx950.
//
// With a residual stream R and a block's output Y, per row of h values:
//   u = Y, or with a norm after the block  u = Y * rstd(Y) * w_post
//   r = R + alpha * gate * u                    (R_out)
//   N = r * rstd(r) * w_pre                     (the next block's input)
//   rstd(x) = 1 / sqrt(mean(x^2) + eps)
// Backward, for the gradients dN of N and dR_out of R_out, with x = R_out * rstd_pre
// and y = Y * rstd_post:
//   d = dN * w_pre,  dr = dR_out + rstd_pre * (d - x * mean(d * x))     (dR)
//   du = alpha * gate * dr
//   dY = du, or  rstd_post * (du * w_post - y * mean(du * w_post * y))
//   dw_pre = sum dN * x,  dw_post = sum du * y,  dgate = sum alpha * dr * u
//
// The second mean needs dr, and so the first: with a = alpha * gate * w_post
//   mean(a y dr) = mean(a y dR_out) + rstd_pre * (mean(a y d) - mean(d x) * mean(a y x)),
// whose four sums are taken together, behind one barrier a row.
//
// Both are HBM streams: every input is read once and every output written once.
// One workgroup holds a whole row in registers (eight values per thread and piece), so
// the means cost no second pass over memory: two workgroup reductions forward, one
// backward.
// The arithmetic is float32; each output is rounded once.  N is formed from the
// float32 r, not from the stored R_out: for a bf16 stream that saves N one rounding.
// Rows need not be 16-byte aligned (any h): gfx950 takes 16-byte global accesses at
// element alignment, at a price, so an odd h's pieces begin on 16 bytes all the same.
//
// Measured: forward 2048 x 8192 bf16 with both norms and a gate 22 us (134 MB, 6.1 TB/s);
// one row of 8192 3.2 us; backward 4096 x 4096 float32 42 us (268 MB, 6.3 TB/s) and 4.3 for
// the sums of the weights' gradients; 1777 x 5003 bf16 26 (107 MB, 4.1 TB/s: ten waves per
// compute unit, and one row ahead does not cover a row's barrier; 30 with two) and 4.5.

#include "norm.h"

namespace ql {
namespace {

// 16, 8 and 4 bytes at any element boundary
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2_any __attribute__((ext_vector_type(2), aligned(4)));

QL_DEV uint16_t nbf16(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }

// How a row divides into pieces of eight values.
//   kWhole   h is a multiple of 8.
//   kEdges   h > 8 is none: pieces begin on 16 bytes, but the first and the last lie wholly
//            inside the row, so that every load is a wide one; they then overlap their
//            neighbours, and count and store only their own values lo .. hi - 1.
//   kTiny    h < 8: one piece, value by value.
enum Rows { kWhole, kEdges, kTiny };

template <Rows K>
struct Cols {
  int c, lo, hi;  // first column; own values; hi == 0: nothing of the row
  // Piece `at` of rows whose first value is `skip` values into a 16-byte piece.
  QL_DEV Cols(int at, int skip, int h) {
    const int raw = 8 * at - skip;
    if (K == kWhole) {
      c = raw;
      lo = 0;
      hi = raw < h ? 8 : 0;
    } else if (K == kEdges) {
      c = raw < 0 ? 0 : raw > h - 8 ? h - 8 : raw;
      lo = raw > h - 8 ? raw - c : 0;
      hi = raw >= h ? 0 : raw < 0 ? 8 + raw : 8;
    } else {
      c = 0;
      lo = 0;
      hi = raw == 0 ? h : 0;
    }
  }
  QL_DEV bool has(int i) const { return K == kWhole || (i >= lo && i < hi); }
  QL_DEV bool whole() const { return K == kWhole || (K == kEdges && lo == 0 && hi == 8); }
};

// Eight values as they are in memory (bf16: 4 registers, float32: 8); zeros where !on.
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  u32x4 v;
  template <Rows K>
  QL_DEV void load(const uint16_t *row, const Cols<K> &q, bool on) {
    v = u32x4{0, 0, 0, 0};
    if (!on || q.hi == 0) return;
    if (K != kTiny) {
      v = *reinterpret_cast<const u32x4_any *>(row + q.c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < q.hi) v[i >> 1] |= (uint32_t)row[i] << (16 * (i & 1));
    }
  }
  QL_DEV float get(int i) const { return (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]); }
};
template <>
struct Piece<float> {
  f32x4 a, b;
  template <Rows K>
  QL_DEV void load(const float *row, const Cols<K> &q, bool on) {
    a = f32x4{0, 0, 0, 0};
    b = f32x4{0, 0, 0, 0};
    if (!on || q.hi == 0) return;
    if (K != kTiny) {
      a = *reinterpret_cast<const f32x4_any *>(row + q.c);
      b = *reinterpret_cast<const f32x4_any *>(row + q.c + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < q.hi) (i < 4 ? a : b)[i & 3] = row[i];
    }
  }
  QL_DEV float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};

template <Rows K>
QL_DEV void store8(uint16_t *row, const float (&x)[8], const Cols<K> &q) {
  if (q.hi == 0) return;
  const u32x4 v{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  if (q.whole()) {
    *reinterpret_cast<u32x4_any *>(row + q.c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (q.has(i)) row[q.c + i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}
template <Rows K>
QL_DEV void store8(float *row, const float (&x)[8], const Cols<K> &q) {
  if (q.hi == 0) return;
  if (q.whole()) {
    *reinterpret_cast<f32x4_any *>(row + q.c) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4_any *>(row + q.c + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (q.has(i)) row[q.c + i] = x[i];
  }
}

// Sum over a wave, the same for every lane: quads, halves and rows of 16 by DPP, then lane
// 15 of a row into the next row and lane 31 into the upper half; lane 63 has the total.
QL_DEV float wave_sum(float v) {
#define QL_DPP(ctrl, rows) \
  __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, rows, 0xF, false))
  v += QL_DPP(0xB1, 0xF);   // quad_perm [1,0,3,2]
  v += QL_DPP(0x4E, 0xF);   // quad_perm [2,3,0,1]
  v += QL_DPP(0x141, 0xF);  // row_half_mirror
  v += QL_DPP(0x140, 0xF);  // row_mirror
  v += QL_DPP(0x142, 0xA);  // row_bcast:15
  v += QL_DPP(0x143, 0xC);  // row_bcast:31
#undef QL_DPP
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

constexpr int kMaxWaves = 16;

// Sum over the workgroup's nw waves, in a fixed order.  One barrier: the callers take the
// four rows of `red` in turn, so a row is written again only after three more barriers,
// when every wave has read it.
QL_DEV float wg_sum(float v, float *red, int nw) {
  v = wave_sum(v);
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kMaxWaves; ++w)
    if (w < nw) v += red[w];
  return v;
}

}  // namespace

// The same for four sums behind one barrier.
QL_DEV f32x4 wg_sum4(f32x4 v, f32x4 *red, int nw) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = wave_sum(v[i]);
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kMaxWaves; ++w)
    if (w < nw) v += red[w];
  return v;
}

// Eight weights; ones where there are none (a product with 1 changes nothing).
template <Rows K>
QL_DEV Piece<float> weights(const float *w, const Cols<K> &q) {
  Piece<float> p;
  if (w) {
    p.load(w, q, true);
  } else {
    p.a = f32x4{1, 1, 1, 1};
    p.b = f32x4{1, 1, 1, 1};
  }
  return p;
}

// Where in a 16-byte piece a workgroup's rows begin (`shift` is 7, or 0 for pieces that
// begin with the row): all its rows are a multiple of 8 apart, so it is one place.
template <Rows K>
QL_DEV int row_skip(int h, int shift) {
  return K == kEdges ? (int)(((int64_t)blockIdx.x * h) & shift) : 0;
}

// NV pieces of eight values per thread, whole waves (8 NV blockDim >= h).  A workgroup walks
// the rows blockIdx.x, + gridDim.x, ...: its weights stay in registers (alpha * gate *
// w_post as one), and the next row is loaded before this one's sums, whose barriers would
// otherwise leave the memory idle.
template <typename RT, int NV, Rows K>
__global__ __launch_bounds__(512) void norm_fwd_kernel(NormFwdArgs p, int shift) {
  __shared__ float red[4][kMaxWaves];
  const int tid = threadIdx.x, B = blockDim.x, nw = B >> 6;
  const int h = (int)p.h, skip = row_skip<K>(h, shift);
  const RT *R = reinterpret_cast<const RT *>(p.R);
  RT *Ro = reinterpret_cast<RT *>(p.R_out);
  const float inv_h = 1.0f / (float)h;
  Piece<float> wp[NV];
  float a[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Cols<K> q(tid + B * j, skip, h);
    const Piece<float> wq = weights(p.w_post, q), wg = weights(p.gate, q);
    wp[j] = weights(p.w_pre, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[j][i] = p.alpha * wg.get(i) * wq.get(i);
  }
  Piece<RT> rr[NV];
  Piece<uint16_t> yy[NV];
  auto load = [&](int64_t m) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols<K> q(tid + B * j, skip, h);
      rr[j].load(R + m * h, q, m < p.M);
      yy[j].load(p.Y + m * h, q, m < p.M && p.Y);
    }
  };
  load(blockIdx.x);
  int slot = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    float r[NV][8], u[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols<K> q(tid + B * j, skip, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[j][i] = q.has(i) ? rr[j].get(i) : 0.0f;
        u[j][i] = q.has(i) ? yy[j].get(i) : 0.0f;
      }
    }
    load(m + gridDim.x);
    if (p.Y) {
      float rs = 1.0f;
      if (p.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(u[j][i], u[j][i], ss);
        rs = 1.0f / sqrtf(wg_sum(ss, red[slot], nw) * inv_h + p.eps);
        slot = (slot + 1) & 3;
        if (p.rstd_post && tid == 0) p.rstd_post[m] = rs;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols<K> q(tid + B * j, skip, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = __builtin_fmaf(a[j][i], u[j][i] * rs, r[j][i]);
        store8(Ro + m * h, r[j], q);
      }
    }
    if (p.w_pre) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(r[j][i], r[j][i], ss);
      const float rs = 1.0f / sqrtf(wg_sum(ss, red[slot], nw) * inv_h + p.eps);
      slot = (slot + 1) & 3;
      if (p.rstd_pre && tid == 0) p.rstd_pre[m] = rs;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols<K> q(tid + B * j, skip, h);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r[j][i] * rs * wp[j].get(i);
        store8(p.N + m * h, o, q);
      }
    }
  }
}

// Backward, rows as above.  The weights' gradients are sums over rows of two products only,
// dN * x and dR * y: w_post's and gate's are constants of the column times the second.  With
// SUMS a workgroup keeps its rows' sums in registers and stores them once, as row blockIdx.x
// of part[2][gridDim.x][h] (norm_sum_kernel adds the rows in a fixed order: no atomics, the
// same bits every time).  The next row is loaded before this one's sums where one piece per
// thread holds a row (h <= 8192); wider rows have no registers left for it.
template <typename RT, int NV, bool SUMS, Rows K>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormBwdArgs p, int shift, float *__restrict__ part) {
  constexpr bool AHEAD = NV == 1;
  __shared__ f32x4 red[4][kMaxWaves];
  const int tid = threadIdx.x, B = blockDim.x, nw = B >> 6;
  const int h = (int)p.h, skip = row_skip<K>(h, shift);
  const RT *Ro = reinterpret_cast<const RT *>(p.R_out), *dRo = reinterpret_cast<const RT *>(p.dR_out);
  RT *dR = reinterpret_cast<RT *>(p.dR);
  const float inv_h = 1.0f / (float)h;
  // this thread's column sums: registers, or with two pieces LDS (they would spill)
  constexpr bool IN_LDS = SUMS && NV == 2;
  __shared__ float sums[IN_LDS ? 2 * NV * 8 * 1024 : 1];
  float s_pre[SUMS && !IN_LDS ? NV : 1][8], s_y[SUMS && !IN_LDS ? NV : 1][8];
  auto sum = [&](int which, int j, int i) -> float & {
    if constexpr (IN_LDS) return sums[((which * NV + j) * 8 + i) * 1024 + tid];
    return which ? s_y[j][i] : s_pre[j][i];
  };
  if constexpr (SUMS)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum(0, j, i) = sum(1, j, i) = 0.0f;
  Piece<float> wp[NV];
  float a[NV][8];  // alpha * gate * w_post
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Cols<K> q(tid + B * j, skip, h);
    const Piece<float> wq = weights(p.w_post, q), wg = weights(p.gate, q);
    wp[j] = weights(p.w_pre, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[j][i] = p.alpha * wg.get(i) * wq.get(i);
  }
  Piece<uint16_t> dn[NV], yy[NV];
  Piece<RT> ro[NV], dro[NV];
  float rsp = 0.0f, rsq = 1.0f;
  auto load = [&](int64_t m) {
    const bool in = m < p.M;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols<K> q(tid + B * j, skip, h);
      dn[j].load(p.dN + m * h, q, in && p.dN);
      ro[j].load(Ro + m * h, q, in && p.w_pre);
      dro[j].load(dRo + m * h, q, in && dRo);
      yy[j].load(p.Y + m * h, q, in && p.Y);
    }
    rsp = in && p.w_pre ? p.rstd_pre[m] : 0.0f;
    rsq = in && p.w_post ? p.rstd_post[m] : 1.0f;
  };
  load(blockIdx.x);
  int slot = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    float d[NV][8], x[NV][8], y[NV][8], dr[NV][8];
    const float rp = rsp, rq = rsq;
    f32x4 sums4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols<K> q(tid + B * j, skip, h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = q.has(i) ? dn[j].get(i) : 0.0f;
        x[j][i] = q.has(i) ? ro[j].get(i) * rp : 0.0f;
        y[j][i] = q.has(i) ? yy[j].get(i) * rq : 0.0f;
        d[j][i] = g * wp[j].get(i);
        dr[j][i] = q.has(i) ? dro[j].get(i) : 0.0f;
        sums4[0] = __builtin_fmaf(d[j][i], x[j][i], sums4[0]);
        if (p.w_post) {  // the second mean's sum in the parts that the first one joins
          const float ay = a[j][i] * y[j][i];
          sums4[1] = __builtin_fmaf(ay, dr[j][i], sums4[1]);
          sums4[2] = __builtin_fmaf(ay, d[j][i], sums4[2]);
          sums4[3] = __builtin_fmaf(ay, x[j][i], sums4[3]);
        }
        if constexpr (SUMS) sum(0, j, i) = __builtin_fmaf(g, x[j][i], sum(0, j, i));
      }
    }
    if (AHEAD) load(m + gridDim.x);
    float mean = 0.0f, mean_post = 0.0f;
    if (p.w_post) {
      sums4 = wg_sum4(sums4, red[slot], nw) * inv_h;
      mean = sums4[0];
      mean_post = sums4[1] + rp * (sums4[2] - mean * sums4[3]);
    } else if (p.w_pre) {
      mean = wg_sum(sums4[0], reinterpret_cast<float *>(red[slot]), nw) * inv_h;
    }
    slot = (slot + 1) & 3;
    if (p.w_pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dr[j][i] += rp * (d[j][i] - x[j][i] * mean);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols<K> q(tid + B * j, skip, h);
      store8(dR + m * h, dr[j], q);
    }
    if (p.dY) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // without a norm after the block y is Y, and the gradient ends here
          if constexpr (SUMS) sum(1, j, i) = __builtin_fmaf(dr[j][i], y[j][i], sum(1, j, i));
          dr[j][i] *= a[j][i];
          if (p.w_post) dr[j][i] = rq * (dr[j][i] - y[j][i] * mean_post);
        }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols<K> q(tid + B * j, skip, h);
        store8(p.dY + m * h, dr[j], q);
      }
    }
    if (!AHEAD) load(m + gridDim.x);
  }
  if constexpr (SUMS) {
    const int64_t plane = (int64_t)gridDim.x * h;
    float *out = part + (int64_t)blockIdx.x * h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols<K> q(tid + B * j, skip, h);
      float v[2][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[0][i] = sum(0, j, i);
        v[1][i] = sum(1, j, i);
      }
      if (p.dw_pre) store8(out, v[0], q);
      if (p.dw_post || p.dgate) store8(out + plane, v[1], q);
    }
  }
}

// Weight gradients from the `rows` partial rows: plane 0 is dw_pre; plane 1, S = sum dR * y,
// gives dw_post = alpha * gate * S and dgate = alpha * w_post * S.  A workgroup takes 64
// columns of a plane; its 16 waves take the rows w, w + 16, ... and are added in wave order.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float *__restrict__ part, int rows, NormBwdArgs p) {
  __shared__ float red[16][64];
  if (blockIdx.y == 0 ? !p.dw_pre : !(p.dw_post || p.dgate)) return;  // the whole workgroup
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t h = p.h, c = (int64_t)blockIdx.x * 64 + l;
  const float *src = part + (int64_t)blockIdx.y * rows * h + c;
  float s = 0.0f;
  if (c < h) {
    int k = w;
    for (; k + 112 < rows; k += 128) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[(int64_t)(k + 16 * i) * h];
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; k < rows; k += 16) s += src[(int64_t)k * h];
  }
  red[w][l] = s;
  __syncthreads();
  if (w == 0 && c < h) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][l];
    if (blockIdx.y == 0) {
      p.dw_pre[c] = s;
    } else {
      if (p.dw_post) p.dw_post[c] = p.alpha * (p.gate ? p.gate[c] : 1.0f) * s;
      if (p.dgate) p.dgate[c] = p.alpha * (p.w_post ? p.w_post[c] : 1.0f) * s;
    }
  }
}

namespace {

// Pieces that a row takes: with h no multiple of 8, up to 7 values before the row's first
// (its pieces then begin on 16 bytes) unless the row fills the workgroup without them.
constexpr int64_t kMaxPieces = kMaxNormWidth / 8;
int row_shift(int64_t h) { return h % 8 && h > 8 && (h + 14) / 8 <= kMaxPieces ? 7 : 0; }
int64_t row_pieces(int64_t h) { return (h + row_shift(h) + 7) / 8; }
// Pieces per thread and threads per row, in whole waves.  Forward, at most 512 threads: two
// rows' workgroups to a compute unit, eight waves at a barrier (2048 x 8192: 21.9 us, with
// 1024 threads of one piece 29 to 32).  Backward, at most 1024: two pieces' operands, sums
// and prefetches take 200 registers, and the compute unit then holds half the threads
// (1777 x 5003: 39 us for 27).
struct RowShape {
  int depth, threads, grid;
};
RowShape row_shape(int64_t M, int64_t h, int most) {
  const int64_t v = row_pieces(h);
  RowShape s;
  s.depth = v <= most ? 1 : v <= 2 * most ? 2 : 4;
  s.threads = (int)((v + 64 * s.depth - 1) / (64 * s.depth) * 64);
  const int64_t fill = 256 * (int64_t)((s.depth == 4 ? 512 : 1024) / s.threads);  // workgroups, a multiple of 8
  s.grid = (int)(M < fill ? M : fill);
  return s;
}
constexpr int kFwdThreads = 512, kBwdThreads = 1024;

template <typename RT, Rows K>
hipError_t fwd(const NormFwdArgs &a, hipStream_t st) {
  const RowShape s = row_shape(a.M, a.h, kFwdThreads);
  const int shift = row_shift(a.h);
  if constexpr (K != kTiny) {
    if (s.depth == 4) return launch(norm_fwd_kernel<RT, 4, K>, s.grid, s.threads, st, a, shift);
    if (s.depth == 2) return launch(norm_fwd_kernel<RT, 2, K>, s.grid, s.threads, st, a, shift);
  }
  return launch(norm_fwd_kernel<RT, 1, K>, s.grid, s.threads, st, a, shift);
}

template <typename RT, bool SUMS, Rows K>
hipError_t bwd(const NormBwdArgs &a, float *part, hipStream_t st) {
  const RowShape s = row_shape(a.M, a.h, kBwdThreads);
  const int shift = row_shift(a.h);
  if constexpr (K != kTiny)
    if (s.depth == 2) return launch(norm_bwd_kernel<RT, 2, SUMS, K>, s.grid, s.threads, st, a, shift, part);
  return launch(norm_bwd_kernel<RT, 1, SUMS, K>, s.grid, s.threads, st, a, shift, part);
}

template <typename RT>
hipError_t fwd_any(const NormFwdArgs &a, hipStream_t st) {
  return a.h % 8 == 0 ? fwd<RT, kWhole>(a, st) : a.h > 8 ? fwd<RT, kEdges>(a, st) : fwd<RT, kTiny>(a, st);
}
template <typename RT, bool SUMS>
hipError_t bwd_any(const NormBwdArgs &a, float *part, hipStream_t st) {
  return a.h % 8 == 0 ? bwd<RT, SUMS, kWhole>(a, part, st)
         : a.h > 8    ? bwd<RT, SUMS, kEdges>(a, part, st)
                      : bwd<RT, SUMS, kTiny>(a, part, st);
}

}  // namespace

size_t norm_bwd_workspace(int64_t M, int64_t h) { return (size_t)2 * row_shape(M, h, kBwdThreads).grid * h * 4; }

hipError_t launch_norm_fwd(const NormFwdArgs &a, bool r_bf16, hipStream_t st) {
  return r_bf16 ? fwd_any<uint16_t>(a, st) : fwd_any<float>(a, st);
}

hipError_t launch_norm_bwd(const NormBwdArgs &a, bool r_bf16, float *part, hipStream_t st) {
  if (!a.dw_pre && !a.dw_post && !a.dgate)
    return r_bf16 ? bwd_any<uint16_t, false>(a, part, st) : bwd_any<float, false>(a, part, st);
  hipError_t e = r_bf16 ? bwd_any<uint16_t, true>(a, part, st) : bwd_any<float, true>(a, part, st);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.h + 63) / 64), 2);
  return launch(norm_sum_kernel, grid, 1024, st, (const float *)part, row_shape(a.M, a.h, kBwdThreads).grid, a);
}

}  // namespace ql
