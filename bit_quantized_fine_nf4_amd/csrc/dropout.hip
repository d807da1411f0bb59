// Inverted dropout of a tensor, for gfx950 (QLoRA trains its adapters with a dropout of
// their input; the linear's fused form is in linear.hip).
//
//   out[e] = bits(e) >= threshold ? x[e] * 65536 / (65536 - threshold) : 0
// with 16 bits per element from a counter-based generator (dropout.h), so the backward
// makes the same decisions again from the same state and no mask is stored.  The scale
// belongs to the probability that 16 bits express, threshold / 65536, which keeps the
// result unbiased.
//
// An HBM stream: eight elements per lane and one generator call (about 60 VALU
// operations, 14 of them 32 x 32 -> 64-bit products) per 32 bytes moved: 2048 x 8192 in
// 10.6 us, 6.3 TB/s, what a copy of that size takes.

#include "dropout.h"

namespace ql {
namespace {

constexpr int kThreads = 256;

QL_DEV float kept(uint32_t bits, uint32_t threshold, float x, float scale) {
  return bits >= threshold ? x * scale : 0.0f;
}
QL_DEV uint16_t dbf16(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }

}  // namespace

__global__ __launch_bounds__(kThreads) void dropout_bf16_kernel(const uint16_t *x, int64_t n, DropState d, float scale,
                                                                uint16_t *out) {
  const uint64_t seed = d.rng[0], offset = d.rng[1];
  const uint32_t t = d.threshold;
  const int64_t nb = (n + 7) >> 3, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < nb; i += stride) {
    if (8 * i + 8 <= n) {
      const u32x4 v = *reinterpret_cast<const u32x4 *>(x + 8 * i);
      const u32x4 w = philox(seed, offset + (uint64_t)i);
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(kept(w[j] & 0xFFFFu, t, bf16_lo(v[j]), scale), kept(w[j] >> 16, t, bf16_hi(v[j]), scale));
      *reinterpret_cast<u32x4 *>(out + 8 * i) = o;
    } else {
      const u32x4 w = philox(seed, offset + (uint64_t)i);
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (8 * i + e < n)
          out[8 * i + e] = dbf16(kept((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu, t,
                                      bf16_lo((uint32_t)x[8 * i + e]), scale));
    }
  }
}

__global__ __launch_bounds__(kThreads) void dropout_f32_kernel(const float *x, int64_t n, DropState d, float scale,
                                                               float *out) {
  const uint64_t seed = d.rng[0], offset = d.rng[1];
  const uint32_t t = d.threshold;
  const int64_t nb = (n + 7) >> 3, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < nb; i += stride) {
    const u32x4 w = philox(seed, offset + (uint64_t)i);
    if (8 * i + 8 <= n) {
      f32x4 a = *reinterpret_cast<const f32x4 *>(x + 8 * i), b = *reinterpret_cast<const f32x4 *>(x + 8 * i + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = kept((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu, t, a[e], scale);
        b[e] = kept((w[2 + (e >> 1)] >> (16 * (e & 1))) & 0xFFFFu, t, b[e], scale);
      }
      *reinterpret_cast<f32x4 *>(out + 8 * i) = a;
      *reinterpret_cast<f32x4 *>(out + 8 * i + 4) = b;
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (8 * i + e < n)
          out[8 * i + e] = kept((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu, t, x[8 * i + e], scale);
    }
  }
}

hipError_t launch_dropout(const void *x, bool bf16, int64_t n, const DropState &d, float scale, void *out,
                          hipStream_t st) {
  const int64_t groups = (n + 8 * kThreads - 1) / (8 * kThreads);
  const unsigned grid = (unsigned)(groups < 4096 ? groups : 4096);  // 16 workgroups per compute unit, then strides
  if (bf16)
    return launch(dropout_bf16_kernel, grid, kThreads, st, reinterpret_cast<const uint16_t *>(x), n, d, scale,
                  reinterpret_cast<uint16_t *>(out));
  return launch(dropout_f32_kernel, grid, kThreads, st, reinterpret_cast<const float *>(x), n, d, scale,
                reinterpret_cast<float *>(out));
}

}  // namespace ql
