// Residual update with RMS norms before and after a block — host interface.
#pragma once

#include "common.h"

namespace ql {

constexpr int64_t kMaxNormWidth = 16384;  // a row stays in one workgroup's registers

struct NormFwdArgs {
  const void *R;        // [M][h] residual stream (float32 or bf16)
  const uint16_t *Y;    // [M][h] bf16 block output, or nullptr
  const float *w_post;  // [h], or nullptr: no norm of Y
  const float *gate;    // [h], or nullptr: 1
  const float *w_pre;   // [h], or nullptr: no N
  float alpha, eps;
  int64_t M, h;
  void *R_out;          // [M][h] (nullptr: not stored; Y == nullptr only)
  uint16_t *N;          // [M][h] bf16
  float *rstd_post, *rstd_pre;  // [M], or nullptr
};

struct NormBwdArgs {
  const uint16_t *dN;   // [M][h] bf16, or nullptr (w_pre == nullptr)
  const void *dR_out;   // [M][h], or nullptr: zero
  const void *R_out;    // [M][h] (w_pre)
  const uint16_t *Y;    // [M][h] bf16 (w_post, or dgate), or nullptr
  const float *rstd_post, *rstd_pre;
  const float *w_post, *gate, *w_pre;
  float alpha;
  int64_t M, h;
  void *dR;             // [M][h]
  uint16_t *dY;         // [M][h] bf16, or nullptr: no block output
  float *dw_pre, *dw_post, *dgate;  // [h], or nullptr
};

size_t norm_bwd_workspace(int64_t M, int64_t h);
hipError_t launch_norm_fwd(const NormFwdArgs &a, bool r_bf16, hipStream_t st);
hipError_t launch_norm_bwd(const NormBwdArgs &a, bool r_bf16, float *part, hipStream_t st);

}  // namespace ql
