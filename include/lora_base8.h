/*
 * lora_base8.h -- C ABI of the operators that train adapters on a frozen base
 * held in 8 bits, by distillation (GB300 / sm_103a): 8-bit blocks of 128, the
 * products of activations and weights held so, and the loss against a teacher's
 * top logits. Same library, status codes and conventions as lora_mlp.h: dense
 * row-major tensors, 16-byte aligned, in the current device's memory; no entry
 * point allocates or synchronises; FP32 sums in a fixed order; a row of an output
 * depends on that row of the inputs (and the weights) only, in every bit; the
 * same bits in every rerun; an argument error launches nothing. Waits that run
 * out are reported by lora_mlp_device_status.
 */
#ifndef LORA_BASE8_H
#define LORA_BASE8_H

#include "lora_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- 8-bit blocks of 128
 * A tensor [M][K] is cut into blocks of `tile` rows x 128 columns (tile 1 for activations
 * and gradients, 128 for weights; the last blocks of a row or column may be smaller), each with an
 * FP32 scale; an e4m3 code c stands for c * scale.
 *   codes   [M][ld] e4m3, ld = K rounded up to a multiple of 16
 *   scales  [ceil(M / tile)][ceil(K / 128)] FP32
 * lora_block8 takes as scale the smallest power of two from 2^-124 to 2^119 of which no
 * value of the block is more than 448 times, and as codes the values / scale rounded to nearest even
 * and held to +-448 (codes past column K: 0). Every value that a code then stands for is a
 * bf16 value exactly. A block that holds a NaN or an infinity has scale NaN and codes 0.
 * The other entry points take any FP32 scales, and do not read codes past column K.
 *   x, out  [M][K] bf16 or fp32; K >= 1, any
 */
lora_status lora_block8(const void *x, int x_type, int tile, int64_t M, int64_t K, void *codes, float *scales,
                        void *stream);
lora_status lora_unblock8(const void *codes, const float *scales, int tile, int64_t M, int64_t K, void *out,
                          int out_type, void *stream);

/* ----------------------------------------- products with weights in 8-bit blocks
 * x [M][K], dy [M][N] in blocks of tile 1, w [N][K] in blocks of tile 128:
 *   forward    y[m][n]  = sum_b (sx[m][b] * sw[n / 128][b]) * (sum of cx[m][k] * cw[n][k], k in block b) + delta[m][n]
 *   backward   dx[m][k] = sum_b (sdy[m][b] * sw[b][k / 128]) * (sum of cdy[m][n] * cw[n][k], n in block b) + delta[m][k]
 * FP32, the blocks' sums added in order, then delta; rounded once to the output's type.
 *   delta  FP32, of the output's size, or NULL (the adapter's delta_y; in the backward pass its dx)
 *   y [M][N], dx [M][K] bf16 or fp32 (out_type)
 * M, K, N < 2^22, any; K, N >= 1.
 */
lora_status lora_block8_linear_fwd(const void *x, const float *x_scales, const void *w, const float *w_scales,
                                   const float *delta, int64_t M, int64_t K, int64_t N, void *y, int out_type,
                                   void *stream);
lora_status lora_block8_linear_bwd(const void *dy, const float *dy_scales, const void *w, const float *w_scales,
                                   const float *delta, int64_t M, int64_t K, int64_t N, void *dx, int out_type,
                                   void *stream);

/* --------------------------------- distillation from a teacher's top logits
 * Row by row, with T = temperature, q = softmax(logits / T) over the V entries of the vocabulary, and the
 * row's entries i: those with ids[i] in [0, V), teacher[i] not -infinity, and no earlier entry of the same id.
 *   p_i  = exp(teacher[i] / T - L)     L = teacher_lse of the row, or log(sum of exp(teacher[i] / T)) when it is NULL
 *   loss = weight * (sum of p_i (log p_i - log q[ids[i]])  [+ r (log r - log rho), with teacher_lse])
 *          r = max(1 - sum of p_i, 0), rho = sum of q over what is no entry; terms of p_i = 0 or r = 0 are 0.
 *          Where rho < 2^-4096, an r of (64 + 8 |teacher_lse|) 2^-24 or less is FP32's rounding of 0 (a teacher that lists all
 *          its mass, a mask that leaves the student nothing else) and counts as 0; a larger one beside rho = 0 is infinite
 *   logits       [M][V] bf16 or fp32 (type)      ids [M][top] int32 or int64 (id_bytes 4 or 8)
 *   teacher      [M][top] bf16 or fp32 (teacher_type)
 *   teacher_lse  [M] FP32, log(sum of exp(t / T)) over the teacher's whole vocabulary, or NULL
 *   weight       [M] FP32, or NULL (all 1). A row of weight 0 is not read: its loss is 0, its gradient 0
 *   loss         [M] FP32 (out)
 *   probs        [M][top] FP32 (out): p_i; -1 for what is no entry, and in rows of weight 0
 *   stats        [M][4] FP32 (out): the largest logit m; log2(sum of exp((logit - m) / T)), with teacher_lse less
 *                log2(max(sum of p_i, 1)); 1 - r / rho (1 without teacher_lse, and where rho < 2^-4096), or,
 *                from r / rho = 2^32 on, -2^32 log2(r / rho); the weight. Zeros in rows of weight 0 or without entries
 * 1 <= V < 2^22, 1 <= top <= 1024, T > 0, finite and no subnormal number. A row without entries has loss 0 and gradient 0.
 */
lora_status lora_distill_topk_fwd(const void *logits, int type, const void *ids, int id_bytes, const void *teacher,
                                  int teacher_type, const float *teacher_lse, const float *weight, float temperature,
                                  int64_t M, int64_t V, int64_t top, float *loss, float *probs, float *stats,
                                  void *stream);

/* Backward pass, the derivative of the loss: dlogits = dloss * weight / T * (P q - p_i at entries, (P - r / rho) q elsewhere),
 * P = 1 or, with teacher_lse, max(sum of p_i, 1) (a teacher's logits of few bits may sum to more than its whole
 * vocabulary's), from the forward's probs and stats (P and the weight among them). Where dloss * weight is 0,
 * and in rows of weight 0 or without entries whatever dloss is, the gradient is 0 and the logits are not read.
 *   dloss    [M] FP32
 *   dlogits  [M][V] of the logits' type, which may be logits itself; or, with scales != NULL, its codes [M][ld]
 *            as lora_block8 would give them for the FP32 values, and scales [M][ceil(V / 128)]
 */
lora_status lora_distill_topk_bwd(const float *dloss, const void *logits, int type, const void *ids, int id_bytes,
                                  const float *probs, const float *stats, float temperature, int64_t M, int64_t V,
                                  int64_t top, void *dlogits, float *scales, void *stream);

#ifdef __cplusplus
}
#endif
#endif
