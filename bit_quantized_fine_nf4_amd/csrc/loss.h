// Softmax cross entropy of an output head without kept logits — host interface.
#pragma once

#include "common.h"

namespace ql {

struct LossArgs {
  const uint16_t *H;      // [M][h] bf16 hidden states
  const uint16_t *W;      // [V][h] bf16 head
  const int64_t *labels;  // [M]; outside [0, V): the token carries no loss
  int64_t M, h, V;        // h a multiple of 64
};

bool loss_supported(int64_t M, int64_t h, int64_t V);
size_t loss_fwd_workspace(int64_t M, int64_t h, int64_t V);
size_t loss_bwd_workspace(int64_t M, int64_t h, int64_t V);
hipError_t launch_loss_fwd(const LossArgs &a, float *loss, float *lse, void *ws, hipStream_t st);
hipError_t launch_loss_bwd(const LossArgs &a, const float *lse, const float *dloss, uint16_t *dH, uint16_t *dW,
                           void *ws, hipStream_t st);

// ---- the products (loss_gemm.hip) ------------------------------------------

// Compact tokens: the n = *count tokens that carry a loss, in order.
struct LogitParams {
  const uint16_t *W;    // rows v0 .. of the head: [nvoc][h]
  const uint16_t *H;    // [n][h] compact hidden states
  const int *count;     // n (device)
  const int *label;     // [n] labels in the whole vocabulary
  int64_t h;
  int64_t v0, nvoc;     // this piece of the vocabulary
  int tiles_v;          // ceil(nvoc / tile rows)
  // statistics: the piece's max and sum of exponentials per tile row of the vocabulary
  f32x2 *part;          // [tiles_v][ldp]
  int64_t ldp;
  float *zlab;          // [n] the label's logit
  // gradient: G = (exp(z - lse) - onehot) * (dloss / top)
  const float *lse, *dloss;  // [n]
  const float *top;          // the largest |dloss| (device)
  uint16_t *G;          // [n][ldg] bf16, ldg = tiles_v * 256; zero past nvoc
  int64_t ldg;
};
// max_tokens bounds n and sizes the grid
hipError_t launch_logit_stats(LogitParams &p, int64_t max_tokens, hipStream_t st);
hipError_t launch_logit_grad(LogitParams &p, int64_t max_tokens, hipStream_t st);
int logit_tile_v(int64_t max_tokens);  // vocabulary rows per statistics tile

struct HeadGradParams {
  const uint16_t *G;   // [n][ldg]
  int64_t ldg;
  const uint16_t *W;   // dH: [nvoc][h] rows of this piece
  const uint16_t *H;   // dW: [n][h] compact hidden states
  const int *count;
  const float *top;    // dW: G's common factor
  int64_t h, nvoc;
  int tiles_m, tiles_n;
  int64_t kper;        // dH: vocabulary entries per split (a multiple of 64)
  float *part;         // dH: [splits][rows][h] float32
  int64_t rows;
  int add;             // dH: add to what part holds (pieces after the first)
  uint16_t *dW;        // dW: [nvoc][h]
};
hipError_t launch_head_dh(HeadGradParams &p, int splits, int64_t max_tokens, hipStream_t st);
hipError_t launch_head_dw(HeadGradParams &p, hipStream_t st);

}  // namespace ql
