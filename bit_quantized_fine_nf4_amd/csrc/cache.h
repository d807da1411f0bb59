// Pages of a key-value cache, and attention of one new token over them — host interface.
#pragma once

#include "common.h"

namespace ql {

// Keys and values lie in pages [pages][hk][page][d] bf16; slot s is token s % page of page
// s / page.
struct CacheShape {
  uint16_t *k, *v;
  int64_t pages;
  int hk, page, d;  // page a power of two in 8..1024, d a multiple of 8 up to 128
};

// rows of K and V [M][hk][d] (token strides ldk, ldv) to their slots; a slot outside the
// cache: its token is not kept
hipError_t launch_cache_write(const CacheShape &c, const uint16_t *K, int64_t ldk, const uint16_t *V, int64_t ldv,
                              const int64_t *slots, int64_t M, hipStream_t st);
// page dst[i] = page src[i]; a pair with a page outside the cache is skipped
hipError_t launch_cache_copy(const CacheShape &c, const int64_t *src, const int64_t *dst, int64_t n, hipStream_t st);

struct DecodeArgs {
  CacheShape c;
  const uint16_t *Q;     // [B][hq][d]
  const int32_t *table;  // [B][width] page of each stretch of `page` tokens
  const int32_t *lens;   // [B] tokens in the cache, the new one included
  const float *slopes;   // [hq], or nullptr
  float scale, cap;      // cap 0: none
  int window;            // 0: all tokens
  int64_t B;
  int hq;
  int64_t width;
  uint16_t *O;           // [B][hq][d]
  void *workspace;       // (nullptr: none needed)
};

size_t decode_workspace(int64_t B, int hq, int hk, int64_t capacity);
hipError_t launch_decode_attn(const DecodeArgs &a, hipStream_t st);

}  // namespace ql
