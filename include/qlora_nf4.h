/*
 * qlora_nf4.h — C ABI of the MI355X (gfx950) NF4 + LoRA linear-layer library.
 *
 * The operations are those of QLoRA as described by
 *   [MC] "QLoRA: Efficient Finetuning of Quantized LLMs" (Michał Chromiak's blog),
 *   [TT] "QLoRA in LLMs" (TensorTonic),
 *   [GO] "QLoRA: the paper that put large-model fine-tuning on a desk" (Good Omens).
 *
 * Conventions shared by every entry point
 *  - Tensor pointers are DEVICE pointers owned by the caller; the library never
 *    allocates, frees or retains them.  Where an entry point needs temporary
 *    device memory the caller passes a workspace sized by qlora_workspace_size().
 *  - `stream` is a hipStream_t (NULL = the default stream).  Every call only
 *    enqueues work and returns without synchronizing; all of a call's work is
 *    ordered on `stream`.  Calls on different streams are safe when their
 *    buffers (workspaces included) are disjoint.
 *  - bf16 tensors are passed as uint16_t bit patterns (bfloat16: 1 sign, 8
 *    exponent, 7 fraction bits).  All matrices are row-major.
 *  - Pointers must be 16-byte aligned unless stated otherwise.
 *  - Errors: arguments are validated before anything is enqueued; on
 *    QLORA_ERR_INVALID_VALUE or QLORA_ERR_UNSUPPORTED nothing is launched and
 *    no output is touched.  A failed kernel launch returns QLORA_ERR_LAUNCH
 *    (kernels of the same call already enqueued before it still run).  The
 *    library takes each launch's status from the launch call itself: it never
 *    reads or clears the calling thread's HIP last-error state, so an error
 *    left there by the caller's own earlier work stays for the caller to see.
 *    No exception crosses the ABI.  Non-finite inputs give unspecified (but
 *    memory-safe) results.
 *  - Thread safety: the library holds no shared mutable state after its
 *    one-time initialisation of the NF4 tables (done under a lock on first
 *    use); the timing hook's events are per thread.
 */
#ifndef QLORA_NF4_H_
#define QLORA_NF4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QLORA_OK = 0,
  QLORA_ERR_INVALID_VALUE = 1, /* bad pointer, size, alignment, rank or workspace */
  QLORA_ERR_UNSUPPORTED = 2,   /* valid request outside what this build supports */
  QLORA_ERR_LAUNCH = 3,        /* the HIP runtime rejected a kernel launch */
  QLORA_ERR_INTERNAL = 4       /* the NF4 tables could not be built */
} qlora_status_t;

typedef enum { QLORA_F32 = 0, QLORA_BF16 = 1 } qlora_dtype_t;

/*
 * 4-bit codebooks.  A code is the index of its value in an ascending 16-entry
 * table (qlora_codebook_levels), chosen as the nearest value to
 * fp32(w / absmax), ties to the lower one.
 *  NF4   the NormalFloat values ([MC] "1. NormalFloat", [TT] §5), code 7 = 0.
 *  INT4  the symmetric absmax integer grid of [TT] §2 at 4 bits: q/7 for
 *        q = -8..7 at code q + 8 (q = -8 is never produced).
 *  FP4   the E2M1 values {0, 0.5, 1, 1.5, 2, 3, 4, 6} and negatives, divided
 *        by 6, at codes 1..15 (code 0, -1.5, is never produced); the pages
 *        compare NF4 with FP4 ([MC] "What the experiments establish") but fix
 *        no FP4 layout, so this one is a reading.
 */
typedef enum { QLORA_CB_NF4 = 0, QLORA_CB_INT4 = 1, QLORA_CB_FP4 = 2 } qlora_codebook_t;

/* Workspace queries (qlora_workspace_size `op`). */
typedef enum {
  QLORA_OP_DOUBLE_QUANT = 0, /* a = number of block scales */
  QLORA_OP_LINEAR_FWD = 1,   /* a = M tokens, b = h, c = o */
  QLORA_OP_LINEAR_BWD = 2,   /* a = M tokens, b = h, c = o */
  QLORA_OP_NORM_BWD = 3,     /* a = M rows, b = h */
  QLORA_OP_LOSS_FWD = 4,     /* a = M tokens, b = h, c = V */
  QLORA_OP_LOSS_BWD = 5,     /* a = M tokens, b = h, c = V */
  QLORA_OP_LINEAR_DROPOUT = 6, /* a = M tokens, b = h, c = o: either direction */
  QLORA_OP_ATTN_BWD = 8,       /* a = M tokens, b = hq, c = hk, r = d */
  QLORA_OP_DECODE_ATTN = 9     /* a = B sequences, b = hq, c = width * page tokens, r = hk */
} qlora_op_t;

#define QLORA_BLOCK 64      /* weights per first-level scale ([MC] "2. Double quantization") */
#define QLORA_CHUNK 256     /* first-level scales per second-level scale ([MC] "A worked memory budget") */
#define QLORA_MAX_RANK 128  /* largest LoRA rank r accepted */

/*
 * One frozen NF4 weight with double-quantized scales.  Logical shape h x o
 * (the pages' W: h inputs, o outputs, [MC] "The algebra").  Stored in
 * PyTorch's Linear.weight order [o][h]: row n holds output n's h weights, so
 * each 64-weight block runs along h.  Produced by qlora_quantize on the [o][h]
 * buffer followed by qlora_double_quant.  This struct is a host object (48
 * bytes on LP64: four pointers, then h at offset 32 and o at offset 40); the
 * pointers in it are device pointers.  Weights encoded with another codebook
 * (qlora_quantize_cb) use the same struct with the `_cb` entry points, which
 * take the codebook as an argument.
 */
typedef struct {
  const uint8_t *codes;   /* h*o/2 bytes: two 4-bit codes per byte, first in the high nibble */
  const int8_t *qabsmax;  /* h*o/64 int8 block scales (mean-centred) */
  const float *scale2;    /* ceil(h*o/64/256) float32 steps, one per 256 block scales */
  const float *mean;      /* 1 float32: the mean of the float32 block scales */
  int64_t h;              /* input width, a positive multiple of 64, at most 2^20 */
  int64_t o;              /* output width, a positive multiple of 64, at most 2^20 */
} qlora_nf4_weight_t;

/*
 * qlora_quantize — blockwise NF4 quantization ([MC] "1. NormalFloat";
 * [TT] §2 "Choose a scale, then round", §3, §5).
 *  w       n weights, float32 or bf16 (w_dtype), any 1-D buffer.
 *  codes   out, ceil(n/2) bytes: code of element 2k in the high nibble of byte k.
 *  absmax  out, ceil(n/64) float32: the largest magnitude of each 64-block.
 * Each weight is divided by its block's largest magnitude (IEEE float32
 * division) and mapped to the nearest of the 16 NF4 levels, ties to the lower
 * level.  A short last block is zero-padded; an odd n pads the last low nibble
 * with code 7 (the zero level); an all-zero block gets code 7 everywhere.
 * Alignment: w 16 bytes; codes and absmax 4 bytes.
 */
qlora_status_t qlora_quantize(const void *w, qlora_dtype_t w_dtype, int64_t n, uint8_t *codes,
                              float *absmax, void *stream);

/*
 * qlora_double_quant — quantization of the block scales ([MC] "2. Double
 * quantization"; [TT] §6; [GO] "Idea two").
 *  absmax   nblocks float32 block scales (from qlora_quantize), all >= 0.
 *  qabsmax  out, nblocks int8.
 *  scale2   out, ceil(nblocks/256) float32 steps.
 *  mean     out, 1 float32 (device).
 *  workspace/ws_bytes  device scratch of at least
 *           qlora_workspace_size(QLORA_OP_DOUBLE_QUANT, nblocks, ...) bytes;
 *           its contents on entry do not matter.
 * mean = the exact mean of all scales rounded once to float32 (independent of
 * summation order).  Each chunk j of 256 consecutive centred scales
 * c = fp32(a - mean) gets step s2_j = fp32(max|c| / 127) and codes
 * q = rint(fp32(c / s2_j)) in [-127, 127] ([TT] §2's symmetric int8 scheme;
 * step 0 gives codes 0).  Requires 1 <= nblocks < 2^32.
 * Alignment: absmax 16 bytes, workspace 256 bytes, qabsmax, scale2 and mean 4.
 */
qlora_status_t qlora_double_quant(const float *absmax, int64_t nblocks, int8_t *qabsmax, float *scale2,
                                  float *mean, void *workspace, size_t ws_bytes, void *stream);

/*
 * qlora_double_quant_noalloc — qlora_double_quant without a workspace, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  Same arguments,
 * results and errors as qlora_double_quant minus workspace/ws_bytes; it
 * allocates nothing and calls no allocating routine.  Its partial sums live in
 * a 48 KB static array the library keeps on each GPU it runs on until the
 * process ends; every accepted size (1 <= nblocks < 2^32) fits in it, since the
 * partial-sum pass never uses more than 512 slots.  The first call on a device
 * looks the array's address up once (hipGetSymbolAddress).  `stream` must
 * belong to the current device (QLORA_ERR_INVALID_VALUE otherwise).  All
 * calls on one GPU share the array: calls that overlap in time on one GPU (on
 * different streams) race and give wrong results; calls ordered on one stream
 * are safe.
 */
qlora_status_t qlora_double_quant_noalloc(const float *absmax, int64_t nblocks, int8_t *qabsmax, float *scale2,
                                          float *mean, void *stream);

/*
 * qlora_dequantize — rebuild n weights ([MC] "1. NormalFloat": codes are
 * dequantized to BF16 for computation; [GO] "The core move").
 *  a_hat = fp32(fp32(qabsmax * scale2) + mean)      (no fused multiply-add)
 *  w_hat = fp32(level[code] * a_hat)                 (out_dtype QLORA_F32)
 *        = bf16 round-to-nearest-even of that value  (out_dtype QLORA_BF16)
 *  out   n float32 or bf16 values.
 * Alignment: codes and out 16 bytes; scale2 and mean 4 bytes; qabsmax any.
 */
qlora_status_t qlora_dequantize(const uint8_t *codes, const int8_t *qabsmax, const float *scale2,
                                const float *mean, int64_t n, void *out, qlora_dtype_t out_dtype,
                                void *stream);

/*
 * Codebook variants of the codec: the same storage, encoder and scales with
 * the levels of `codebook` (qlora_quantize / qlora_dequantize are the
 * QLORA_CB_NF4 cases).  Arguments, layouts and alignment as above.
 */
qlora_status_t qlora_quantize_cb(const void *w, qlora_dtype_t w_dtype, int64_t n, qlora_codebook_t codebook,
                                 uint8_t *codes, float *absmax, void *stream);
qlora_status_t qlora_dequantize_cb(const uint8_t *codes, const int8_t *qabsmax, const float *scale2,
                                   const float *mean, int64_t n, qlora_codebook_t codebook, void *out,
                                   qlora_dtype_t out_dtype, void *stream);

/*
 * qlora_dequantize_nodq — reconstruction without double quantization: the
 * float32 block scales from quantization are used as stored,
 * w_hat = fp32(level[code] * absmax[block]) ([MC] "2. Double quantization"
 * is an addition on top of blockwise quantization).  absmax 4-byte aligned.
 */
qlora_status_t qlora_dequantize_nodq(const uint8_t *codes, const float *absmax, int64_t n,
                                     qlora_codebook_t codebook, void *out, qlora_dtype_t out_dtype,
                                     void *stream);

/* The 16 float32 values of a codebook, ascending (index = code). */
qlora_status_t qlora_codebook_levels(qlora_codebook_t codebook, float *levels);

/*
 * qlora_linear_fwd — Y = X·W_hat + s·(X·L1)·L2 ([MC] "The algebra", Eq. 3;
 * [TT] §3), with W_hat the bf16 dequantization of W computed on the fly.
 *  X   [M][h] bf16.     L1 [h][r] bf16.    L2 [r][o] bf16.
 *  Y   out [M][o] bf16.
 *  T   out [M][r] bf16 = X·L1 (float32 accumulation, rounded once), kept for
 *      the backward pass.
 *  r = 0 means no adapter: L1, L2 and T may be NULL.  1 <= M, 0 <= r <= 128.
 *  workspace: qlora_workspace_size(QLORA_OP_LINEAR_FWD, M, h, o, r) bytes.
 * Products accumulate in float32 on bf16 operands; outputs round once to bf16.
 */
qlora_status_t qlora_linear_fwd(const qlora_nf4_weight_t *W, const uint16_t *X, int64_t M,
                                const uint16_t *L1, const uint16_t *L2, int32_t r, float s,
                                uint16_t *Y, uint16_t *T, void *workspace, size_t ws_bytes,
                                void *stream);

/*
 * qlora_linear_bwd — gradients through the frozen dequantized weight into the
 * adapters ([MC] Figure 1 and "One training step"; [TT] §4; [GO] "The core
 * move": no gradient ever updates the 4-bit weights, so there is no dW).
 *  With U = dY·L2^T:
 *   dX  = dY·W_hat^T + s·U·L1^T   out [M][h] bf16
 *   dL1 = s·X^T·U                 out [h][r] float32
 *   dL2 = s·T^T·dY                out [r][o] float32
 *  T is the forward's saved [M][r] bf16 product X·L1.  r = 0: only dX is
 *  computed and X, T, L1, L2, dL1, dL2 may be NULL.
 *  workspace: qlora_workspace_size(QLORA_OP_LINEAR_BWD, M, h, o, r) bytes.
 *  The token sum behind dL1 and dL2 is split into chunks whose operand rows
 *  stay below 2^31 bytes each; a shape that would need more than 65535 such
 *  chunks (only for M in the hundreds of millions on the widest layers)
 *  returns QLORA_ERR_UNSUPPORTED.
 */
qlora_status_t qlora_linear_bwd(const qlora_nf4_weight_t *W, const uint16_t *X, const uint16_t *T,
                                const uint16_t *dY, int64_t M, const uint16_t *L1, const uint16_t *L2,
                                int32_t r, float s, uint16_t *dX, float *dL1, float *dL2,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * The linear layer on a weight encoded with another codebook
 * (qlora_quantize_cb): arguments, layouts and errors as qlora_linear_fwd and
 * qlora_linear_bwd, the codes decoded with the levels of `codebook`
 * (qlora_linear_fwd / qlora_linear_bwd are the QLORA_CB_NF4 cases).
 */
qlora_status_t qlora_linear_fwd_cb(const qlora_nf4_weight_t *W, qlora_codebook_t codebook, const uint16_t *X,
                                   int64_t M, const uint16_t *L1, const uint16_t *L2, int32_t r, float s,
                                   uint16_t *Y, uint16_t *T, void *workspace, size_t ws_bytes, void *stream);
qlora_status_t qlora_linear_bwd_cb(const qlora_nf4_weight_t *W, qlora_codebook_t codebook, const uint16_t *X,
                                   const uint16_t *T, const uint16_t *dY, int64_t M, const uint16_t *L1,
                                   const uint16_t *L2, int32_t r, float s, uint16_t *dX, float *dL1, float *dL2,
                                   void *workspace, size_t ws_bytes, void *stream);

/*
 * Dropout from a counter-based generator, with a mask that is never stored (the pages'
 * adapter configuration, [TT] "LoraConfig", sets lora_dropout = 0.05 beside r and alpha).
 * Element e of a tensor has 16 random bits: the (e % 8)-th 16-bit piece, low half of a
 * word first, of Philox4x32-7 (Salmon et al., 2011) with key `seed` and the 128-bit
 * counter (offset + e / 8, 0).  It is kept when its bits reach t = rint(65536 p); kept
 * values are scaled by 65536 / (65536 - t), which is unbiased at the probability t / 65536
 * that 16 bits express.  A dropped element is 0 whatever it held.
 *  p    0 <= p < 1 with t <= 65535.
 *  rng  DEVICE pointer to two uint64: {seed, offset}, 8-byte aligned, read when the call
 *       runs: a captured graph advances the offset between replays by writing there.
 *       A forward and its backward take the same state; the next use of n elements takes
 *       an offset at least ceil(n / 8) further.
 *
 * qlora_dropout  out[e] = dropout of x[e], n elements of float32 or bf16 (one rounding).
 *  The same call on a gradient is the backward.  out may be x.  16-byte aligned.
 *
 * qlora_linear_fwd_dropout / qlora_linear_bwd_dropout — the linear layer with dropout on
 * its adapter's input: element (m, k) of X is element m*h + k.  With s' = s / (1 - t/65536)
 * and keep the 0/1 mask:
 *   T = (keep ⊙ X)·L1                 Y  = X·W_hat + s'·T·L2
 *   U = dY·L2^T                       dX = dY·W_hat^T + s'·keep ⊙ (U·L1^T)
 *   dL1 = s'·(keep ⊙ X)^T·U           dL2 = s'·T^T·dY
 *  T (bf16, without the scale) is the forward's output for the backward.  dL1 keeps U to
 *  float32's 24 bits.  The frozen part sees all of X.  W_hat is the bf16 dequantization at
 *  every M.  Where nothing is dropped (t = 0) Y and dX are the plain linear's, which for
 *  M <= 16 rounds the levels to bf16 and applies the block scales to sums (Y) or to dY in
 *  bf16 (dX).  Other arguments, layouts and errors as qlora_linear_fwd_cb and
 *  qlora_linear_bwd_cb; r = 0 is the plain linear.
 *  workspace: qlora_workspace_size(QLORA_OP_LINEAR_DROPOUT, M, h, o, r) bytes.
 */
qlora_status_t qlora_dropout(const void *x, qlora_dtype_t dtype, int64_t n, double p, const uint64_t *rng, void *out,
                             void *stream);
qlora_status_t qlora_linear_fwd_dropout(const qlora_nf4_weight_t *W, qlora_codebook_t codebook, const uint16_t *X,
                                        int64_t M, const uint16_t *L1, const uint16_t *L2, int32_t r, float s,
                                        double p, const uint64_t *rng, uint16_t *Y, uint16_t *T, void *workspace,
                                        size_t ws_bytes, void *stream);
qlora_status_t qlora_linear_bwd_dropout(const qlora_nf4_weight_t *W, qlora_codebook_t codebook, const uint16_t *X,
                                        const uint16_t *T, const uint16_t *dY, int64_t M, const uint16_t *L1,
                                        const uint16_t *L2, int32_t r, float s, double p, const uint64_t *rng,
                                        uint16_t *dX, float *dL1, float *dL2, void *workspace, size_t ws_bytes,
                                        void *stream);

/*
 * qlora_merge_adapter — merge a trained adapter into the frozen base
 * ([TT] §11 "Saving, Loading, and Merging QLoRA Adapters": dequantize the base
 * to a wider precision and add the LoRA update; [GO] "What it added up to").
 *  W' = W_hat + s·L1·L2 in W's [o][h] storage: entry (n, k) =
 *       fp32(w_hat + fp32(s * P)),  P = sum_q L1[k][q] * L2[q][n]
 *  where w_hat is qlora_dequantize's float32 value and P comes from bf16
 *  products with float32 accumulation (summation order unspecified).
 *  L1 [h][r] bf16, L2 [r][o] bf16, 16-byte aligned (may be NULL when r = 0),
 *       0 <= r <= 128.
 *  out  [o][h] float32 or bf16 (round to nearest even of the float32 value);
 *       16-byte aligned.
 */
qlora_status_t qlora_merge_adapter(const qlora_nf4_weight_t *W, const uint16_t *L1, const uint16_t *L2,
                                   int32_t r, float s, void *out, qlora_dtype_t out_dtype, void *stream);

/*
 * qlora_merge_requantize — the merge followed by NF4 re-quantization in one
 * pass ([TT] §11: merging and quantizing again adds a second quantization
 * error).  codes_out (h*o/2 bytes) and absmax_out (h*o/64 float32) are what
 * qlora_quantize returns for the float32 merged weight qlora_merge_adapter
 * computes; follow with qlora_double_quant(absmax_out, ...) to obtain the new
 * weight's int8 scales.  codes_out 8-byte and absmax_out 4-byte aligned; they must not
 * alias W's buffers.
 */
qlora_status_t qlora_merge_requantize(const qlora_nf4_weight_t *W, const uint16_t *L1, const uint16_t *L2,
                                      int32_t r, float s, uint8_t *codes_out, float *absmax_out, void *stream);

/*
 * The merge and the merge with re-quantization for a weight encoded with
 * another codebook: W_hat uses the levels of `codebook` and the re-encoding
 * uses the same codebook.  Otherwise as qlora_merge_adapter and
 * qlora_merge_requantize (the QLORA_CB_NF4 cases).
 */
qlora_status_t qlora_merge_adapter_cb(const qlora_nf4_weight_t *W, qlora_codebook_t codebook, const uint16_t *L1,
                                      const uint16_t *L2, int32_t r, float s, void *out, qlora_dtype_t out_dtype,
                                      void *stream);
qlora_status_t qlora_merge_requantize_cb(const qlora_nf4_weight_t *W, qlora_codebook_t codebook, const uint16_t *L1,
                                         const uint16_t *L2, int32_t r, float s, uint8_t *codes_out,
                                         float *absmax_out, void *stream);

/*
 * qlora_adamw_step — one optimizer step on adapter parameters ([TT] §4 "One
 * QLoRA Training Step, End to End": only the adapters are updated; the update
 * itself is not written out on the pages, so this is AdamW with decoupled
 * weight decay, Loshchilov and Hutter).  Elementwise over n float32 values:
 *   p <- p * (1 - lr*wd)
 *   m <- beta1*m + (1 - beta1)*g          v <- beta2*v + (1 - beta2)*g*g
 *   p <- p - lr/(1 - beta1^t) * m / (sqrt(v)/sqrt(1 - beta2^t) + eps)
 *  param      float32 master values, updated in place (e.g. L1 then L2, flat)
 *  grad       float32 gradients (qlora_linear_bwd's dL1 / dL2)
 *  exp_avg, exp_avg_sq   float32 first / second moments, updated in place;
 *             start at 0 before step 1.  Like param and grad they may live in
 *             device memory or in pinned host memory allocated with
 *             hipHostMalloc (optimizer state kept in CPU RAM, [TT] §7 "Paged
 *             Optimizers"; the kernel then reads and writes it over the link).
 *  step       t, 1-based.   0 <= beta1, beta2 < 1;  eps > 0;  lr, wd >= 0.
 *  param_bf16 optional (may be NULL): receives bf16(p) (round to nearest even),
 *             the copy the linear layer consumes.
 *  param, grad, exp_avg, exp_avg_sq 16-byte aligned, param_bf16 8-byte aligned;
 *  no two of the arrays may overlap.
 */
qlora_status_t qlora_adamw_step(float *param, const float *grad, float *exp_avg, float *exp_avg_sq, int64_t n,
                                int64_t step, float lr, float beta1, float beta2, float eps, float weight_decay,
                                uint16_t *param_bf16, void *stream);

/*
 * Block glue: the elementwise steps between the NF4 linears of a transformer
 * block.  [MC] "A closer look: Design choices and memory costs" puts adapters
 * on every linear of the block, attention and feed-forward; the feed-forward of
 * the LLaMA models the pages name is gated, its gate and up projections G and
 * U meeting in H = SiLU(G) * U with SiLU(g) = g / (1 + exp(-g)) before the down
 * projection.  All tensors are n bf16 values in any matching shape, 16-byte
 * aligned; arithmetic is float32, each output rounded once to nearest even.
 * Outputs must not overlap the inputs (qlora_grad_sum excepted, see there).
 *
 * qlora_silu_gate_fwd  H = SiLU(G) * U.
 * qlora_silu_gate_bwd  for the upstream gradient dH:
 *                        dU = dH * SiLU(G)
 *                        dG = dH * U * sigmoid(G) * (1 + G * (1 - sigmoid(G)))
 *                      dG and dU must be different buffers.
 * qlora_grad_sum       out = parts[0] + ... + parts[k-1], summed in that order:
 *                      the gradient of an input that several linears read (the
 *                      block input feeds q, k, v, gate and up).  `parts` is a
 *                      HOST array of k device pointers, 1 <= k <= 8; `out` may
 *                      be one of them (exactly, not a partial overlap).
 */
qlora_status_t qlora_silu_gate_fwd(const uint16_t *G, const uint16_t *U, int64_t n, uint16_t *H, void *stream);
qlora_status_t qlora_silu_gate_bwd(const uint16_t *G, const uint16_t *U, const uint16_t *dH, int64_t n, uint16_t *dG,
                                   uint16_t *dU, void *stream);
qlora_status_t qlora_grad_sum(const uint16_t *const *parts, int32_t k, int64_t n, uint16_t *out, void *stream);

/*
 * Norms before and after a block, fused with the block's gate and residual scale.
 * The pages' linears sit in the blocks of a LLaMA-like transformer ([MC] "A closer
 * look: Design choices and memory costs"); between two blocks the residual stream R
 * takes the block's output Y and is normalised for the next block.  With
 * rstd(x) = 1 / sqrt(mean(x^2) + eps) over a row of h values:
 *   u     = Y, or Y * rstd(Y) * w_post where the block has a norm after it
 *   R_out = R + alpha * gate * u
 *   N     = R_out * rstd(R_out) * w_pre
 * Arithmetic is float32 and each output is rounded once; N is formed from the
 * float32 R_out, before it is rounded to a bf16 stream.  M rows, 1 <= h <= 16384
 * (any h; a wider row, or more than 2^40 values, is QLORA_ERR_UNSUPPORTED).  Y, N,
 * dN and dY are [M][h] bf16; the stream (R, R_out, dR_out, dR) is [M][h] of r_dtype;
 * weights, gate and their gradients are [h] float32, rstd_post and rstd_pre [M]
 * float32.  All pointers are 16-byte aligned.  Squares of magnitudes above 1e18 overflow float32: rows that
 * hold such values give unspecified results, like non-finite ones.
 *
 * qlora_norm_fwd
 *  Y       may be NULL (the norm before the first block): then w_post and gate are
 *          NULL, R_out is R itself and its pointer may be NULL or R (not stored).
 *  w_post  NULL: no norm after the block.   gate  NULL: 1.   alpha  finite.
 *  w_pre   NULL: no N (the residual update alone); N and rstd_pre are not used.
 *  R_out   may be R (in place).  rstd_post and rstd_pre may be NULL (inference);
 *          they are what the backward takes.  At least one of Y and w_pre is given.
 *
 * qlora_norm_bwd   for the gradients dN of N and dR_out of R_out, with
 *   x = R_out * rstd_pre,  d = dN * w_pre,  y = Y * rstd_post:
 *     dR   = dR_out + rstd_pre * (d - x * mean(d * x))         (the gradient of R)
 *     dY   = alpha * gate * dR, or with a norm after the block, du being that:
 *            rstd_post * (du * w_post - y * mean(du * w_post * y))
 *     dw_pre = sum dN * x    dw_post = sum du * y    dgate = sum alpha * dR * u
 *  (dR enters the later lines in float32.)
 *  w_pre   NULL: no N; dN, R_out, rstd_pre and dw_pre are not used and dR = dR_out.
 *  dR_out  NULL: zero (only with w_pre).   dR may be dR_out (in place).
 *  dY      NULL: there was no block output; Y, w_post, gate, dw_post, dgate are NULL.
 *  Y       needed with w_post and with dgate.
 *  dw_pre, dw_post, dgate   NULL: that weight is frozen.  The sums over rows run in
 *          a fixed order (no atomics).
 *  workspace: qlora_workspace_size(QLORA_OP_NORM_BWD, M, h, 0, 0) bytes, 256-byte
 *          aligned, needed only when one of the three is wanted.
 */
qlora_status_t qlora_norm_fwd(const void *R, qlora_dtype_t r_dtype, const uint16_t *Y, const float *w_post,
                              const float *gate, float alpha, const float *w_pre, float eps, int64_t M, int64_t h,
                              void *R_out, uint16_t *N, float *rstd_post, float *rstd_pre, void *stream);
qlora_status_t qlora_norm_bwd(const uint16_t *dN, const void *dR_out, qlora_dtype_t r_dtype, const void *R_out,
                              const uint16_t *Y, const float *rstd_post, const float *rstd_pre, const float *w_post,
                              const float *gate, float alpha, const float *w_pre, int64_t M, int64_t h, void *dR,
                              uint16_t *dY, float *dw_pre, float *dw_post, float *dgate, void *workspace,
                              size_t ws_bytes, void *stream);

/*
 * Softmax cross entropy of an output head over a large vocabulary, with its gradient
 * ([MC] "One training step", [TT] §4 "One QLoRA Training Step, End to End": forward,
 * loss, backward).  For hidden states H [M][h] bf16, a head W [V][h] bf16 (a linear's
 * weight order) and labels [M] int64, with z = H·W^T in float32:
 *   lse  = log(sum_v exp(z_v))            loss = lse - z[label]
 *   G    = (exp(z - lse) - onehot(label)) * dloss
 *   dH   = G·W                            dW   = G^T·H
 * z is never stored.  The forward keeps per-tile statistics; the backward computes z
 * again in pieces of the vocabulary, each turned into bf16 G (one rounding, then
 * float32 sums) in the workspace.  A token whose label is outside [0, V), such as
 * -100, carries no loss: its loss and lse are 0, its dH row is 0, it adds nothing to
 * dW, costs no products (but where all tokens are one tile), and its H row may hold
 * anything.  Sums run in a fixed order.
 *  A word whose logit is -inf (a masked one) has probability 0, whole tiles of them too.
 *  M, V >= 1, h a positive multiple of 64.  h > 2^20, M or V > 2^24, or more than
 *  2^24 tiles of 256 tokens x 128 words are QLORA_ERR_UNSUPPORTED.
 *  H, W, dH, dW 16-byte aligned; labels 8; loss, lse, dloss 4; workspace 256.
 *
 * qlora_loss_fwd  loss, lse   out, [M] float32.
 *  workspace: qlora_workspace_size(QLORA_OP_LOSS_FWD, M, h, V, 0) bytes.
 * qlora_loss_bwd  lse as the forward gave it; dloss [M] float32, the gradient of each
 *  token's loss (1 / count for the mean).  dH out, [M][h] bf16.  dW out, [V][h] bf16,
 *  or NULL: the head is frozen.  Outputs overlap nothing.  A dloss that is not finite
 *  makes its own token's dH not finite, and dW; the other tokens' dH are as without it.
 *  workspace: qlora_workspace_size(QLORA_OP_LOSS_BWD, M, h, V, 0) bytes.
 */
qlora_status_t qlora_loss_fwd(const uint16_t *H, const uint16_t *W, const int64_t *labels, int64_t M, int64_t h,
                              int64_t V, float *loss, float *lse, void *workspace, size_t ws_bytes, void *stream);
qlora_status_t qlora_loss_bwd(const uint16_t *H, const uint16_t *W, const int64_t *labels, const float *lse,
                              const float *dloss, int64_t M, int64_t h, int64_t V, uint16_t *dH, uint16_t *dW,
                              void *workspace, size_t ws_bytes, void *stream);

/*
 * Rotary positions of queries and keys.  The pages' linears include a block's q, k, v and o
 * projections ([MC] "A closer look: Design choices and memory costs"); what lies between
 * them is the attention of a LLaMA-like transformer: rotary positions, attention, and for
 * answering a cache of keys and values.
 *
 * qlora_rope  Pair i of the first `rot` values of every head turns by the angle
 *   t = positions[m] * freqs[i]:  (a, b) -> scale * (a cos t - b sin t, a sin t + b cos t).
 *  The angle is formed in float64, the rest in float32, each output rounded once; the
 *  values past `rot` are copied.  A position is exact in float64 (below 2^53).
 *  Q       [M][hq][d] bf16: token m's heads start at Q + m * ldq.   ldq >= hq * d.
 *  K       [M][hk][d] likewise, or NULL with hk = 0: one tensor only.
 *  positions  M int64 (8-byte aligned).   freqs  rot / 2 float64 radians per position, on
 *          the device (8-byte aligned; qlora_rope_freqs makes them).
 *  interleaved  0: pairs (i, i + rot / 2); 1: pairs (2 i, 2 i + 1).
 *  inverse  1: turns back by t, which with the same scale is the gradient of the forward.
 *  Q_out, K_out  with token strides ldqo, ldko; either may be its input with the same
 *          stride (in place), and overlaps nothing else.
 *  d a multiple of 8 up to 256; rot even, 2 <= rot <= d; strides multiples of 8; tensors
 *  16-byte aligned.  M > 2^23, heads > 4096 in all or strides > 2^21 are
 *  QLORA_ERR_UNSUPPORTED.
 *
 * qlora_rope_freqs  (host) the radians per position of each pair, base^(-2 i / rot), and
 *  the scale, for contexts `factor` times the `original` length:
 *   QLORA_ROPE_NONE    as they are.          QLORA_ROPE_LINEAR  divided by the factor.
 *   QLORA_ROPE_NTK     with the base times factor^(rot / (rot - 2)).
 *   QLORA_ROPE_YARN    (Peng et al., 2023) pairs that turn `slow` times or less over the
 *                      original length divided by the factor, those that turn `fast` times
 *                      or more as they are, in proportion between; scale 0.1 ln(factor) + 1.
 *  freqs   out, rot / 2 doubles on the host.  scale  out, 1 unless YARN.
 *  base > 1, factor >= 1; original >= 1 and fast > slow for YARN (otherwise unused).
 */
typedef enum { QLORA_ROPE_NONE = 0, QLORA_ROPE_LINEAR = 1, QLORA_ROPE_NTK = 2, QLORA_ROPE_YARN = 3 } qlora_rope_t;

qlora_status_t qlora_rope_freqs(int32_t rot, double base, qlora_rope_t scaling, double factor, double original,
                                double slow, double fast, double *freqs, float *scale);
qlora_status_t qlora_rope(const uint16_t *Q, int64_t ldq, int32_t hq, const uint16_t *K, int64_t ldk, int32_t hk,
                          const int64_t *positions, const double *freqs, float scale, int32_t interleaved,
                          int32_t inverse, int64_t M, int32_t d, int32_t rot, uint16_t *Q_out, int64_t ldqo,
                          uint16_t *K_out, int64_t ldko, void *stream);

/*
 * Attention of packed tokens, each query over one span of keys.  With spans[i] = (lo, hi),
 * query i sees the keys lo <= j < hi (clamped to [0, M); none if lo >= hi):
 *   z_ij = scale * q_i . k_j        cap > 0:  z <- cap * tanh(z / cap), off by roundings of z
 *                                   slopes:   z <- z - slopes[head] * |i - j|
 *   O_i  = sum_j softmax(z_i)_j v_j,   lse_i = log sum_j exp(z_ij)
 * A query that sees nothing has O = 0, lse = -inf, passes no gradient, and its rows of Q,
 * O, lse and dO may hold anything.  What a query does not see does not enter its results,
 * infinities and NaN included.  A NaN that a query holds or sees in a key makes its row of O
 * and its lse NaN; an infinity or NaN that it sees in a value leaves that column of its row of
 * O not finite.
 * Query head h reads key head h / (hq / hk).
 *  Q [M][hq][d], K and V [M][hk][d] bf16 with token strides ldq, ldk, ldv; O, dO and the
 *  gradients are dense.  lse [hq][M] float32.  spans M x 2 int32, slopes hq float32 or NULL.
 *  scale > 0, cap 0 (none) or more; either (but a cap of 0) outside 2^-60..2^60 is
 *  QLORA_ERR_UNSUPPORTED.  d a multiple of 8 up to 128, strides multiples of 8, hq a multiple of hk;
 *  bf16 tensors and lse 16-byte aligned, spans 8, slopes 4.  Products are of bf16 operands
 *  with float32 sums: the softmax weights and score gradients are rounded to bf16 for the
 *  products that follow.  M > 2^24, hq > 4096, 2^24 or more stretches of 128 queries in all
 *  heads, or strides > 2^21 are QLORA_ERR_UNSUPPORTED.
 *
 * qlora_attn_spans  the spans of packed documents.  documents  n + 1 int32 on the device,
 *  not decreasing: document e has the tokens documents[e] <= i < documents[e + 1]; tokens
 *  of no document see nothing.  causal 1: a token sees its document up to itself, and the
 *  first prefix[e] tokens of its document (prefix: n int32 on the device, or NULL: 0);
 *  causal 0: all of its document (prefix not used).  window > 0: no token further than
 *  window - 1 back, nor, without causal, further ahead; a prefix is seen ahead whatever the window.
 *
 * qlora_attn_bwd  the gradients of Q, K and V for the gradient dO of O, with O and lse as
 *  the forward gave them (of Q, K, V, spans, scale, cap and slopes as given to it).  Sums
 *  run in a fixed order.  dK and dV are summed over the query heads of their key head.  What
 *  is not finite in a query, its dO or a key or value that it sees leaves the gradients that
 *  the formulas make of it not finite, and no others.
 *  A query's D = sum_j softmax(z)_j (dO . v_j) is dO . O with the bf16 O, or, if it sees at most
 *  256 keys or its head's |slope| is 1/16 or more, that sum: by its own span and head alone.
 *  workspace: qlora_workspace_size(QLORA_OP_ATTN_BWD, M, hq, hk, d) bytes, 256-byte aligned.
 */
qlora_status_t qlora_attn_spans(const int32_t *documents, int64_t n, const int32_t *prefix, int64_t M, int32_t causal,
                                int64_t window, int32_t *spans, void *stream);
qlora_status_t qlora_attn_fwd(const uint16_t *Q, int64_t ldq, const uint16_t *K, int64_t ldk, const uint16_t *V,
                              int64_t ldv, const int32_t *spans, const float *slopes, float scale, float cap, int64_t M,
                              int32_t hq, int32_t hk, int32_t d, uint16_t *O, float *lse, void *stream);
qlora_status_t qlora_attn_bwd(const uint16_t *dO, const uint16_t *Q, int64_t ldq, const uint16_t *K, int64_t ldk,
                              const uint16_t *V, int64_t ldv, const uint16_t *O, const float *lse,
                              const int32_t *spans, const float *slopes, float scale, float cap, int64_t M, int32_t hq,
                              int32_t hk, int32_t d, uint16_t *dQ, uint16_t *dK, uint16_t *dV, void *workspace,
                              size_t ws_bytes, void *stream);

/*
 * A cache of keys and values in pages: k and v are each [pages][hk][page][d] bf16, 16-byte
 * aligned, page a power of two in 8..1024, d a multiple of 8 up to 128.  Token t of page p
 * has the slot p * page + t.  Which pages a sequence has, and which are free, is the
 * caller's: the entry points read page numbers from device memory and skip those that are
 * not in the cache.
 *
 * qlora_cache_write  rows of K and V ([M][hk][d], token strides ldk and ldv, multiples of 8)
 *  to the slots of their tokens (M int64); a token whose slot is outside the cache is not
 *  kept.  Slots of one call are distinct (the values left in one that is named twice are
 *  unspecified); other slots keep what they hold.
 * qlora_cache_copy  page dst[i] = page src[i] for n pairs (int64): a fork or a compaction.
 *  A pair with a page outside the cache is skipped.  No dst of a call is another's dst or
 *  src (otherwise the pages concerned are left unspecified).
 * qlora_decode_attn  attention of one new token for each of B sequences over its tokens in
 *  the cache, the new one's own key and value among them (written before):
 *    O = sum_j softmax(z)_j v_j over max(0, n - window) <= j < n (window 0: from 0), n = lens[b],
 *  z, cap, slopes, heads and types as qlora_attn_fwd, the query standing at n - 1.
 *   Q, O    [B][hq][d], dense.   table  [B][width] int32: the page of tokens page * e ..
 *   lens    B int32, clamped to 0..width * page; 0 gives O = 0.
 *  Tokens whose page is not in the cache count as masked.  Pages and tokens that a sequence
 *  does not see are not read.  NaN and infinities that it sees reach O as in qlora_attn_fwd.
 *  workspace: qlora_workspace_size(QLORA_OP_DECODE_ATTN, B, hq, width * page, hk) bytes,
 *  256-byte aligned (0: not needed).
 *  More than 2^30 slots or 2^30 tokens of capacity (width * page), M > 2^31, n > 2^23,
 *  B * hq > 2^20, hq > 4096 or strides > 2^21 are QLORA_ERR_UNSUPPORTED.
 */
qlora_status_t qlora_cache_write(const uint16_t *K, int64_t ldk, const uint16_t *V, int64_t ldv, const int64_t *slots,
                                 int64_t M, uint16_t *k_pages, uint16_t *v_pages, int64_t pages, int32_t hk,
                                 int32_t page, int32_t d, void *stream);
qlora_status_t qlora_cache_copy(uint16_t *k_pages, uint16_t *v_pages, int64_t pages, int32_t hk, int32_t page,
                                int32_t d, const int64_t *src, const int64_t *dst, int64_t n, void *stream);
qlora_status_t qlora_decode_attn(const uint16_t *Q, const uint16_t *k_pages, const uint16_t *v_pages, int64_t pages,
                                 int32_t page, const int32_t *table, int64_t width, const int32_t *lens,
                                 const float *slopes, float scale, float cap, int64_t window, int64_t B, int32_t hq,
                                 int32_t hk, int32_t d, uint16_t *O, void *workspace, size_t ws_bytes, void *stream);

/* Workspace bytes an entry point needs (always a multiple of 256; may be 0).  Sizes past
 * an entry point's limits give its QLORA_ERR_UNSUPPORTED here too. */
qlora_status_t qlora_workspace_size(qlora_op_t op, int64_t a, int64_t b, int64_t c, int32_t r,
                                    size_t *bytes);

/*
 * Timing hook for benchmarks and profilers.  `kernel` 0 = the forward fused
 * dequant-GEMM, 1 = the dX kernel of qlora_linear_bwd (the fused dequant-GEMM,
 * or for M <= 16 the few-token dX kernel), 2 = the few-token forward
 * (M <= 16).  When `start`/`stop` (hipEvent_t handles) are non-NULL, every
 * later launch of that kernel by the calling thread records `start` just
 * before and `stop` just after itself on the call's stream.  NULL/NULL turns
 * the hook off.  Per thread; the library only records, never synchronizes.
 * Events created with hipEventDisableSystemFence disturb the timed stream
 * least (a default event's system-scope fence stalls it for microseconds).
 */
qlora_status_t qlora_set_timing_events(int32_t kernel, void *start, void *stop);

/*
 * Stream probe, a measurement helper rather than a step of the method: the
 * plain HBM streaming rate for the byte mix of a bandwidth-bound kernel, the
 * ceiling its own rate is compared with.  Moves `n_tiles` tiles; tile t reads
 * the 1024 * rd contiguous bytes of `src` at byte 1024 * rd * t and writes the
 * 1024 * wr contiguous bytes of `dst` at byte 1024 * wr * t, with fully
 * coalesced 16-byte accesses.  Launch shape: `blocks` workgroups of 256
 * threads (0: min(ceil(n_tiles / 8), 8192); at most 2^20), each wave taking
 * `depth` tiles (1, 2, 4 or 8) per pass with all their loads issued first; a
 * caller takes the best rate over a sweep of shapes as the ceiling.
 *   (rd, wr) = (1, 0)  read only (the few-token forward's weight stream);
 *              (4, 1)  four bytes read per byte written (quantization of bf16
 *                      weights reads 2 and writes 0.52 bytes per weight);
 *              (1, 4)  the reverse (dequantization to bf16).
 *  src: n_tiles * 1024 * rd bytes; dst: n_tiles * 1024 * wr bytes, or 16 bytes
 *  when wr = 0 (it may receive one store).  Both 16-byte aligned.  The values
 *  written are a function of those read and otherwise unspecified.
 *  QLORA_ERR_INVALID_VALUE for any other (rd, wr) or depth, blocks out of
 *  range, NULL or misaligned pointers, or n_tiles < 1.
 */
qlora_status_t qlora_stream_probe(int32_t rd, int32_t wr, int32_t depth, int32_t blocks, const void *src, void *dst,
                                  int64_t n_tiles, void *stream);

/* Static description of a status code (never NULL). */
const char *qlora_status_string(qlora_status_t status);

/* Host copy of the 16 float32 NF4 levels the kernels use, ascending
 * (code 0 = -1, code 7 = 0, code 15 = +1).  Returns QLORA_ERR_INTERNAL if the
 * tables could not be built. */
qlora_status_t qlora_nf4_levels(float out[16]);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_NF4_H_ */
