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
// Both are HBM streams: every input is read once and every output written once.
// One workgroup holds a whole row in registers (eight values per thread and piece),
// so the two means cost two workgroup reductions and no second pass over memory.
// The arithmetic is float32; each output is rounded once.  N is formed from the
// float32 r, not from the stored R_out: for a bf16 stream that saves N one rounding.
// Rows need not be 16-byte aligned (any h): gfx950 takes 16-byte global accesses at
// element alignment; a row's last h % 8 values go one by one.

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

// Eight values as they are in memory (bf16: 4 registers, float32: 8).  TAIL: h is not
// a multiple of 8, and a row's last piece has n < 8 values, taken as 4, 2 and 1 of them
// and zeros after them.
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  u32x4 v;
  template <bool TAIL>
  QL_DEV void load(const uint16_t *p, int n) {
    v = u32x4{0, 0, 0, 0};
    if (TAIL ? n >= 8 : n > 0) {
      v = *reinterpret_cast<const u32x4_any *>(p);
    } else if (TAIL && n > 0) {
      const bool four = n & 4, two = n & 2;
      const uint32_t b = two ? *reinterpret_cast<const u32_any *>(p + (n & 4)) : 0u;
      const uint32_t c = (n & 1) ? p[n & 6] : 0u;
      if (four) {
        const u32x2 a = *reinterpret_cast<const u32x2_any *>(p);
        v = u32x4{a[0], a[1], two ? b : c, two ? c : 0u};
      } else {
        v = u32x4{two ? b : c, two ? c : 0u, 0u, 0u};
      }
    }
  }
  QL_DEV float get(int i) const { return (i & 1) ? bf16_hi(v[i >> 1]) : bf16_lo(v[i >> 1]); }
};
template <>
struct Piece<float> {
  f32x4 a, b;
  template <bool TAIL>
  QL_DEV void load(const float *p, int n) {
    a = f32x4{0, 0, 0, 0};
    b = f32x4{0, 0, 0, 0};
    if (TAIL ? n >= 8 : n > 0) {
      a = *reinterpret_cast<const f32x4_any *>(p);
      b = *reinterpret_cast<const f32x4_any *>(p + 4);
    } else if (TAIL && n > 0) {
      f32x4 t = f32x4{0, 0, 0, 0};
      const float one = (n & 1) ? p[n & 6] : 0.0f;
      if (n & 2) {
        const f32x2 w = *reinterpret_cast<const f32x2_any *>(p + (n & 4));
        t = f32x4{w[0], w[1], one, 0};
      } else {
        t[0] = one;
      }
      if (n & 4) {
        a = *reinterpret_cast<const f32x4_any *>(p);
        b = t;
      } else {
        a = t;
      }
    }
  }
  QL_DEV float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};

template <bool TAIL>
QL_DEV void store8(uint16_t *p, const float (&x)[8], int n) {
  const u32x4 v{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  if (!TAIL || n >= 8) {
    *reinterpret_cast<u32x4_any *>(p) = v;
  } else {
    if (n & 4) *reinterpret_cast<u32x2_any *>(p) = u32x2{v[0], v[1]};
    const uint32_t b = (n & 4) ? v[2] : v[0], c = (n & 2) ? ((n & 4) ? v[3] : v[1]) : b;
    if (n & 2) *reinterpret_cast<u32_any *>(p + (n & 4)) = b;
    if (n & 1) p[n & 6] = (uint16_t)c;
  }
}
template <bool TAIL>
QL_DEV void store8(float *p, const float (&x)[8], int n) {
  const f32x4 a{x[0], x[1], x[2], x[3]}, b{x[4], x[5], x[6], x[7]};
  if (!TAIL || n >= 8) {
    *reinterpret_cast<f32x4_any *>(p) = a;
    *reinterpret_cast<f32x4_any *>(p + 4) = b;
  } else {
    if (n & 4) *reinterpret_cast<f32x4_any *>(p) = a;
    const f32x4 t = (n & 4) ? b : a;
    if (n & 2) *reinterpret_cast<f32x2_any *>(p + (n & 4)) = f32x2{t[0], t[1]};
    if (n & 1) p[n & 6] = (n & 2) ? t[2] : t[0];
  }
}

// Sum over the workgroup of B threads, in a fixed order; `red` has B / 64 floats that
// nobody reads or writes until the barrier of the call after the next one.
template <int B>
QL_DEV float wg_sum(float v, float *red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  if constexpr (B > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < B / 64; ++w) v += red[w];
  }
  return v;
}

}  // namespace

// B threads per row, NV pieces of eight values per thread (8 B NV >= h).
template <typename RT, int B, int NV, bool TAIL>
__global__ __launch_bounds__(B) void norm_fwd_kernel(NormFwdArgs p) {
  __shared__ float red[4][B / 64];
  const int tid = threadIdx.x;
  const int h = (int)p.h;
  const RT *R = reinterpret_cast<const RT *>(p.R);
  RT *Ro = reinterpret_cast<RT *>(p.R_out);
  const float inv_h = 1.0f / (float)h;
  int slot = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    float r[NV][8];
    Piece<RT> rr[NV];
    Piece<uint16_t> yy[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (tid + B * j);
      rr[j].template load<TAIL>(R + m * h + (c < h ? c : 0), c < h ? h - c : 0);
      if (p.Y) yy[j].template load<TAIL>(p.Y + m * h + (c < h ? c : 0), c < h ? h - c : 0);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) r[j][i] = rr[j].get(i);
    if (p.Y) {
      float rs = 1.0f;
      if (p.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(yy[j].get(i), yy[j].get(i), ss);
        rs = 1.0f / sqrtf(wg_sum<B>(ss, red[slot]) * inv_h + p.eps);
        slot = (slot + 1) & 3;
        if (p.rstd_post && tid == 0) p.rstd_post[m] = rs;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j);
        if (c >= h) continue;
        Piece<float> w, g;
        if (p.w_post) w.template load<TAIL>(p.w_post + c, h - c);
        if (p.gate) g.template load<TAIL>(p.gate + c, h - c);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float u = yy[j].get(i);
          if (p.w_post) u = u * rs * w.get(i);
          const float a = p.gate ? p.alpha * g.get(i) : p.alpha;
          r[j][i] = __builtin_fmaf(a, u, r[j][i]);
          o[i] = r[j][i];
        }
        store8<TAIL>(Ro + m * h + c, o, h - c);
      }
    } else if (Ro) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j);
        if (c < h) store8<TAIL>(Ro + m * h + c, r[j], h - c);
      }
    }
    if (p.w_pre) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(r[j][i], r[j][i], ss);
      const float rs = 1.0f / sqrtf(wg_sum<B>(ss, red[slot]) * inv_h + p.eps);
      slot = (slot + 1) & 3;
      if (p.rstd_pre && tid == 0) p.rstd_pre[m] = rs;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j);
        if (c >= h) continue;
        Piece<float> w;
        w.template load<TAIL>(p.w_pre + c, h - c);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r[j][i] * rs * w.get(i);
        store8<TAIL>(p.N + m * h + c, o, h - c);
      }
    }
  }
}

// Backward.  A workgroup takes the rows blockIdx.x, + gridDim.x, ...; with SUMS it
// keeps its rows' contributions to the three weight gradients in registers and
// stores them once, as row blockIdx.x of part[3][gridDim.x][h] (norm_sum_kernel adds
// the rows in a fixed order: no atomics, the same bits every time).
template <typename RT, int B, int NV, bool SUMS, bool TAIL>
__global__ __launch_bounds__(B) void norm_bwd_kernel(NormBwdArgs p, float *__restrict__ part) {
  __shared__ float red[4][B / 64];
  const int tid = threadIdx.x;
  const int h = (int)p.h;
  const RT *Ro = reinterpret_cast<const RT *>(p.R_out), *dRo = reinterpret_cast<const RT *>(p.dR_out);
  RT *dR = reinterpret_cast<RT *>(p.dR);
  const float inv_h = 1.0f / (float)h;
  constexpr int NS = SUMS ? NV : 1;
  float s_pre[NS][8], s_post[NS][8], s_gate[NS][8];
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[j][i] = s_post[j][i] = s_gate[j][i] = 0.0f;
  int slot = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    Piece<uint16_t> dn[NV], yy[NV];
    Piece<RT> ro[NV], dro[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (tid + B * j), n = c < h ? h - c : 0;
      const int64_t at = m * h + (n ? c : 0);
      dn[j].template load<TAIL>(p.dN ? p.dN + at : nullptr, p.dN ? n : 0);
      ro[j].template load<TAIL>(p.w_pre ? Ro + at : nullptr, p.w_pre ? n : 0);
      dro[j].template load<TAIL>(dRo ? dRo + at : nullptr, dRo ? n : 0);
      yy[j].template load<TAIL>(p.Y ? p.Y + at : nullptr, p.Y ? n : 0);
    }
    float dr[NV][8];
    if (p.w_pre) {
      const float rs = p.rstd_pre[m];
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j);
        Piece<float> w;
        w.template load<TAIL>(p.w_pre + (c < h ? c : 0), c < h ? h - c : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = ro[j].get(i) * rs, d = dn[j].get(i) * w.get(i);
          dr[j][i] = d;
          dot = __builtin_fmaf(d, x, dot);
          if (SUMS) s_pre[SUMS ? j : 0][i] = __builtin_fmaf(dn[j].get(i), x, s_pre[SUMS ? j : 0][i]);
        }
      }
      dot = wg_sum<B>(dot, red[slot]) * inv_h;
      slot = (slot + 1) & 3;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dr[j][i] = dro[j].get(i) + rs * (dr[j][i] - ro[j].get(i) * rs * dot);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dr[j][i] = dro[j].get(i);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (tid + B * j);
      if (c < h) store8<TAIL>(dR + m * h + c, dr[j], h - c);
    }
    if (!p.dY) continue;
    if (p.w_post) {
      const float rs = p.rstd_post[m];
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j), n = c < h ? h - c : 0;
        Piece<float> w, g;
        w.template load<TAIL>(p.w_post + (n ? c : 0), n);
        if (p.gate) g.template load<TAIL>(p.gate + (n ? c : 0), n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = yy[j].get(i) * rs;
          const float adr = p.alpha * dr[j][i], du = p.gate ? adr * g.get(i) : adr, d = du * w.get(i);
          if (SUMS) {
            s_post[SUMS ? j : 0][i] = __builtin_fmaf(du, y, s_post[SUMS ? j : 0][i]);
            s_gate[SUMS ? j : 0][i] = __builtin_fmaf(adr, y * w.get(i), s_gate[SUMS ? j : 0][i]);
          }
          dot = __builtin_fmaf(d, y, dot);
          dr[j][i] = d;
        }
      }
      dot = wg_sum<B>(dot, red[slot]) * inv_h;
      slot = (slot + 1) & 3;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j);
        if (c >= h) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rs * (dr[j][i] - yy[j].get(i) * rs * dot);
        store8<TAIL>(p.dY + m * h + c, o, h - c);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (tid + B * j);
        if (c >= h) continue;
        Piece<float> g;
        if (p.gate) g.template load<TAIL>(p.gate + c, h - c);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float adr = p.alpha * dr[j][i];
          o[i] = p.gate ? adr * g.get(i) : adr;
          if (SUMS) s_gate[SUMS ? j : 0][i] = __builtin_fmaf(adr, yy[j].get(i), s_gate[SUMS ? j : 0][i]);
        }
        store8<TAIL>(p.dY + m * h + c, o, h - c);
      }
    }
  }
  if constexpr (SUMS) {
    const int64_t plane = (int64_t)gridDim.x * h;
    float *out = part + (int64_t)blockIdx.x * h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (tid + B * j);
      if (c >= h) continue;
      if (p.dw_pre) store8<TAIL>(out + c, s_pre[j], h - c);
      if (p.dw_post) store8<TAIL>(out + plane + c, s_post[j], h - c);
      if (p.dgate) store8<TAIL>(out + 2 * plane + c, s_gate[j], h - c);
    }
  }
}

// out[k][c] = sum of the `rows` partial rows of weight gradient k = blockIdx.y.  A
// workgroup takes 64 columns; its 16 waves take the rows w, w + 16, ... and are added
// in wave order.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float *__restrict__ part, int rows, int64_t h,
                                                        float *dw_pre, float *dw_post, float *dgate) {
  __shared__ float red[16][64];
  float *out = blockIdx.y == 0 ? dw_pre : (blockIdx.y == 1 ? dw_post : dgate);
  if (!out) return;  // the whole workgroup
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + l;
  const float *src = part + (int64_t)blockIdx.y * rows * h + c;
  float s = 0.0f;
  if (c < h) {
    int k = w;
    for (; k + 48 < rows; k += 64) {
      const float a = src[(int64_t)k * h], b = src[(int64_t)(k + 16) * h];
      const float d = src[(int64_t)(k + 32) * h], e = src[(int64_t)(k + 48) * h];
      s += (a + b) + (d + e);
    }
    for (; k < rows; k += 16) s += src[(int64_t)k * h];
  }
  red[w][l] = s;
  __syncthreads();
  if (w == 0 && c < h) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][l];
    out[c] = s;
  }
}

namespace {

// Rows of partial sums: one workgroup per compute unit for rows of 1024 threads and
// proportionally more of the smaller ones.
int bwd_grid(int64_t M, int64_t h) {
  const int64_t per = h <= 2048 ? 1024 : (h <= 4096 ? 512 : 256);
  return (int)(M < per ? M : per);
}

template <typename RT, bool TAIL>
hipError_t fwd(const NormFwdArgs &a, hipStream_t st) {
  const int64_t v = (a.h + 7) / 8;
  const unsigned grid = (unsigned)(a.M < (1 << 20) ? a.M : (1 << 20));
  if (v <= 64) return launch(norm_fwd_kernel<RT, 64, 1, TAIL>, grid, 64, st, a);
  if (v <= 256) return launch(norm_fwd_kernel<RT, 256, 1, TAIL>, grid, 256, st, a);
  if (v <= 512) return launch(norm_fwd_kernel<RT, 512, 1, TAIL>, grid, 512, st, a);
  if (v <= 1024) return launch(norm_fwd_kernel<RT, 1024, 1, TAIL>, grid, 1024, st, a);
  return launch(norm_fwd_kernel<RT, 1024, 2, TAIL>, grid, 1024, st, a);
}

template <typename RT, bool SUMS, bool TAIL>
hipError_t bwd(const NormBwdArgs &a, float *part, hipStream_t st) {
  const int64_t v = (a.h + 7) / 8;
  const unsigned grid = SUMS ? (unsigned)bwd_grid(a.M, a.h) : (unsigned)(a.M < (1 << 20) ? a.M : (1 << 20));
  if (v <= 64) return launch(norm_bwd_kernel<RT, 64, 1, SUMS, TAIL>, grid, 64, st, a, part);
  if (v <= 256) return launch(norm_bwd_kernel<RT, 256, 1, SUMS, TAIL>, grid, 256, st, a, part);
  if (v <= 512) return launch(norm_bwd_kernel<RT, 512, 1, SUMS, TAIL>, grid, 512, st, a, part);
  if (v <= 1024) return launch(norm_bwd_kernel<RT, 1024, 1, SUMS, TAIL>, grid, 1024, st, a, part);
  return launch(norm_bwd_kernel<RT, 1024, 2, SUMS, TAIL>, grid, 1024, st, a, part);
}

template <typename RT>
hipError_t fwd_any(const NormFwdArgs &a, hipStream_t st) {
  return a.h % 8 ? fwd<RT, true>(a, st) : fwd<RT, false>(a, st);
}
template <typename RT, bool SUMS>
hipError_t bwd_any(const NormBwdArgs &a, float *part, hipStream_t st) {
  return a.h % 8 ? bwd<RT, SUMS, true>(a, part, st) : bwd<RT, SUMS, false>(a, part, st);
}

}  // namespace

size_t norm_bwd_workspace(int64_t M, int64_t h) { return (size_t)3 * bwd_grid(M, h) * h * 4; }

hipError_t launch_norm_fwd(const NormFwdArgs &a, bool r_bf16, hipStream_t st) {
  return r_bf16 ? fwd_any<uint16_t>(a, st) : fwd_any<float>(a, st);
}

hipError_t launch_norm_bwd(const NormBwdArgs &a, bool r_bf16, float *part, hipStream_t st) {
  if (!a.dw_pre && !a.dw_post && !a.dgate)
    return r_bf16 ? bwd_any<uint16_t, false>(a, part, st) : bwd_any<float, false>(a, part, st);
  hipError_t e = r_bf16 ? bwd_any<uint16_t, true>(a, part, st) : bwd_any<float, true>(a, part, st);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.h + 63) / 64), 3);
  return launch(norm_sum_kernel, grid, 1024, st, (const float *)part, bwd_grid(a.M, a.h), a.h, a.dw_pre, a.dw_post,
                a.dgate);
}

}  // namespace ql
