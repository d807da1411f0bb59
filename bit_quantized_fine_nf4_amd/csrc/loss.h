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
  const uint16_t *H;    // [n][h] compact hidden states, blocked
  const int *count;     // n (device)
  const int *label;     // [n] labels in the whole vocabulary
  int64_t h;
  int64_t v0, nvoc;     // this piece of the vocabulary
  int tiles_v;          // ceil(nvoc / tile rows)
  // statistics: max and sum of exponentials per 128 vocabulary rows (sum 0: no rows)
  f32x2 *part;          // [ceil(nvoc / 128), even for 256-row tiles][ldp]
  int64_t ldp;
  float *zlab;          // [n] the label's logit
  // statistics of at most kFewTokens tokens without a compact copy (labels set): H is all
  // tokens' hidden states, [M][h] as they are
  const int64_t *labels;  // [M]
  int64_t M;
  // gradient: G = (exp(z - lse) - onehot) * (dloss / top)
  const float *lse, *dloss;  // [n]
  const float *top;          // the largest finite |dloss| (device)
  uint16_t *G;          // [n][piece], blocked, gblocks blocks per row; zero past nvoc up to
  int64_t gblocks;      // the next 256 and past n up to the next 32
};
constexpr int kFewTokens = 32;
hipError_t launch_logit_stats_few(LogitParams &p, hipStream_t st);
// max_tokens bounds n and chooses the tiles
hipError_t launch_logit_stats(LogitParams &p, int64_t max_tokens, hipStream_t st);
hipError_t launch_logit_grad(LogitParams &p, int64_t max_tokens, hipStream_t st);
hipError_t launch_logit_wide(LogitParams &p, bool grad, hipStream_t st);  // 256 x 256 tiles
bool logits_wide(int64_t max_tokens, int64_t h, int64_t nvoc);
int logit_parts(int64_t max_tokens, int64_t h, int64_t V);  // rows of part

struct HeadGradParams {
  const uint16_t *G;   // [n][piece], blocked
  int64_t gblocks;     // blocks per row
  const uint16_t *W;   // dH: [nvoc][h] rows of this piece
  const uint16_t *H;   // dW: [n][h] compact hidden states, blocked
  const int *count;
  const float *top;    // dW: G's common factor
  int64_t h, nvoc;
  int tiles_n;
  int64_t first;       // dH: entries of the first piece, which set the splits
  int64_t kper;        // dH for at most 64 tokens: vocabulary entries per split
  float *part;         // dH: [splits][n][h] float32 (at most 64 tokens: [splits][rows][h])
  int64_t rows;        // rows of h that part has room for in all (at most 64 tokens: M)
  int add;             // dH: add to what part holds (pieces after the first)
  uint16_t *dW;        // dW: [nvoc][h]
};
hipError_t launch_head_dh(HeadGradParams &p, int64_t max_tokens, hipStream_t st);
hipError_t launch_head_dh_wide(HeadGradParams &p, hipStream_t st);
hipError_t launch_head_dw(HeadGradParams &p, hipStream_t st);

// Splits of dH's sum over a piece of the vocabulary, for n tokens on 256 x 256 tiles: the
// count in 1..16 that leaves the 256 persistent workgroups idle the least, counting a
// split's partial sums as 4 % of a round of whole tiles.  Host and device choose alike: n
// is known on the device only.  `rows`: how many rows of partial sums there is room for.
__host__ __device__ inline int head_splits(int64_t n, int64_t h, int64_t piece, int64_t rows) {
  const int64_t tiles = (n + 255) / 256 * ((h + 255) / 256), blocks = (piece + 63) / 64;
  int best = 1;
  int64_t cost = 0;
  for (int s = 1; s <= 16 && (s == 1 || (blocks >= 8 * s && s * n <= rows)); ++s) {
    // rounds of 1 / s tile each, in units of 1 / 10000 of a tile
    const int64_t c = (tiles * s + 255) / 256 * 10000 / s + 400 * s * tiles / 256;
    if (s == 1 || c < cost) cost = c, best = s;
  }
  return best;
}

}  // namespace ql
