// Dropout from a counter-based generator: the generator for the kernels, and the host
// interface of the elementwise dropout.
#pragma once

#include "common.h"

namespace ql {

// Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011; 7 rounds are the fewest its authors found to pass every test
// of their batteries).  Key: the 64-bit seed.  Counter: 64 bits, the upper half zero.
// One call makes 128 bits, 16 for each of eight consecutive elements: element e has the
// (e % 8)-th 16-bit piece (low half of a word first) of counter offset + e / 8.
QL_DEV u32x4 philox(uint64_t seed, uint64_t counter) {
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  uint32_t x0 = (uint32_t)counter, x1 = (uint32_t)(counter >> 32), x2 = 0, x3 = 0;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
    x1 = (uint32_t)b;
    x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
    x3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{x0, x1, x2, x3};
}

// The seed and offset of a call, read from the device so that a captured graph can
// advance them, and the drop threshold: an element is kept when its 16 bits reach it.
struct DropState {
  const uint64_t *rng;  // {seed, offset}
  uint32_t threshold;   // 0..65535
};

// Eight bf16 values (elements 8 block .. 8 block + 7) with the dropped ones zeroed.
// A select, not a product: a dropped NaN or infinity is gone.
QL_DEV u32x4 drop8(u32x4 x, uint64_t seed, uint64_t counter, uint32_t threshold) {
  const u32x4 w = philox(seed, counter);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = (w[j] & 0xFFFFu) >= threshold ? 0xFFFFu : 0u;
    const uint32_t hi = (w[j] >> 16) >= threshold ? 0xFFFF0000u : 0u;
    x[j] &= lo | hi;
  }
  return x;
}

// The same eight decisions as bits (element i: bit i).
QL_DEV uint32_t keep_bits(uint64_t seed, uint64_t counter, uint32_t threshold) {
  const u32x4 w = philox(seed, counter);
  uint32_t b = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    b |= ((w[j] & 0xFFFFu) >= threshold ? 1u << (2 * j) : 0u) | ((w[j] >> 16) >= threshold ? 2u << (2 * j) : 0u);
  return b;
}

// out = x * scale where kept, else 0; out may be x.
hipError_t launch_dropout(const void *x, bool bf16, int64_t n, const DropState &d, float scale, void *out,
                          hipStream_t st);

}  // namespace ql
