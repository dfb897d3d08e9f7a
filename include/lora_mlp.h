/*
 * lora_mlp.h -- C ABI of the operators around the LoRA delta in an MLP block
 * (GB300 / sm_103a): layer norm, activation checkpoints in 8 bits and their use
 * in the backward pass, and the gated feed-forward block. Same library, status
 * codes and conventions as lora_delta.h:
 *   - Tensors are dense, row-major, contiguous, in the current device's memory
 *     (the Python functions refuse those of another one), 16-byte aligned. The
 *     caller owns every buffer and the stream; no entry point allocates or
 *     synchronises (the status calls at the end excepted). A workspace needs no
 *     initial value (lora_delta_bwd_packed8's excepted).
 *   - Sizes below 2^31, M >= 0. M = 0 returns LORA_OK; gradients that are sums
 *     over the rows are then written as zeros, nothing else is.
 *   - Every sum is FP32 in a fixed order that does not depend on the device. A
 *     row of an output with M rows depends on that row of the inputs only, in
 *     every bit (batch invariance); sums over the rows are the same bits in
 *     every rerun. No atomics.
 *   - An argument error (also an unknown type, activation or kind code:
 *     LORA_ERR_SHAPE) launches nothing.
 */
#ifndef LORA_MLP_H
#define LORA_MLP_H

#include "lora_delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { LORA_BF16 = 0, LORA_F32 = 1 };

/* ------------------------------------------------------------- layer norm
 *   mean = sum(x) / N    var = sum((x - mean)^2) / N    rstd = 1 / sqrt(var + eps)
 *   y = (x - mean) * rstd * weight + bias
 *   x       [M][N] bf16 or fp32 (x_type)      y  [M][N] of x_type (out)
 *   weight, bias  [N] bf16 or fp32 (w_type); bias may be NULL (no bias)
 *   mean, rstd    [M] fp32 (out), kept for the backward pass
 * N >= 1, any. NaN and infinity in a row reach that row's outputs only.
 */
lora_status lora_layer_norm_fwd(const void *x, int x_type, const void *weight, const void *bias, int w_type, float eps,
                                int64_t M, int64_t N, void *y, float *mean, float *rstd, void *stream);

/* Backward pass, xh = (x - mean) * rstd, g = dy * weight:
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh))    dw = sum_m dy * xh    db = sum_m dy
 *   dy, dx  [M][N] of `type`; dw, db [N] fp32 (db may be NULL: not wanted)
 *   x       [M][N] of `type` when x_scales is NULL; otherwise the 8-bit codes of a
 *           packed x (lora_pack8, [M][32 ceil(N / 32)]) and x_scales its scale bytes
 */
size_t lora_layer_norm_bwd_workspace_size(int64_t M, int64_t N);
lora_status lora_layer_norm_bwd(const void *dy, int type, const void *x, const void *x_scales, const void *weight,
                                int w_type, const float *mean, const float *rstd, int64_t M, int64_t N, void *dx,
                                float *dw, float *db, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------- activation checkpoints in 8 bits
 * A row is cut into groups of 32 elements (the last one padded with zeros), each with a
 * scale 2^(s - 127), s its scale byte, and 32 codes c (signed 8 bits, |c| <= 127), standing
 * for c * 2^(s - 127): s is the smallest for which the group's largest magnitude is at most
 * 127.5 steps (at most 248, so that no value overflows); c is x / step rounded to nearest
 * even, held to +-127. Every value it stands for is a bf16 value exactly, so a consumer that takes
 * bf16 operands loses nothing more. A group that holds a NaN or an infinity has s = 255, and all its
 * values read NaN.
 *   x       [M][K] bf16 or fp32; K >= 1, any
 *   codes   [M][32 G] int8, scales [M][G] uint8, G = ceil(K / 32)
 */
lora_status lora_pack8(const void *x, int x_type, int64_t M, int64_t K, void *codes, void *scales, void *stream);
lora_status lora_unpack8(const void *codes, const void *scales, int64_t M, int64_t K, void *out, int out_type,
                         void *stream);

/* dA = du^T @ x of a packed x: da [R][K] fp32, du [M][R] bf16. K a multiple of 8, R of 8 in
 * [8, 64]. Bit for bit the dA that lora_delta_bwd gives for the unpacked x. */
size_t lora_pack8_da_workspace_size(int64_t M, int64_t K, int64_t R);
lora_status lora_pack8_da(const void *du, const void *codes, const void *scales, int64_t M, int64_t K, int64_t R,
                          float *da, void *workspace, size_t workspace_bytes, void *stream);

/* lora_delta_bwd with x given packed: same outputs, bit for bit those of lora_delta_bwd for
 * the unpacked x, which is nowhere formed (M = 0, where that call writes nothing: da and db are
 * written as zeros, as everywhere here). The workspace starts with lora_delta_bwd's control block
 * (zero before its first use), whose status block its kernels report to. */
size_t lora_delta_bwd_packed8_workspace_size(int64_t M, int64_t K, int64_t N, int64_t R);
lora_status lora_delta_bwd_packed8(const void *dy, const void *codes, const void *scales, const void *a, const void *b,
                                   const void *u, float alpha, int64_t M, int64_t K, int64_t N, int64_t R, float *dx,
                                   float *da, float *db, void *du, void *workspace, size_t workspace_bytes,
                                   void *stream);

/* ------------------------------------------------ gated feed-forward block
 *   G = x Wg^T + Dg    U = x Wu^T + Du    h = act(G) * U           (FP32, h rounded to bf16 once)
 *   x [M][K], w_gate, w_up [F][K] bf16; h [M][F] bf16 (out); K and F multiples of 8; M, K, F < 2^22
 *   delta_gate, delta_up  Dg, Du [M][F] fp32 (the delta_y of two LoRA sites), or both NULL
 *   act   silu: y / (1 + exp(-y)), or gelu in its tanh form
 *   keep  what is kept of G and U for the backward pass: nothing (the four pointers are ignored),
 *         bf16 [M][F], or packed as lora_pack8 would pack their FP32 values (codes and scales)
 * Backward, from the kept G and U:
 *   dU = dh * act(G)   dG = dh * U * act'(G)   (rounded to bf16: dup, dgate [M][F], out)
 *   dx = dG Wg + dU Wu [M][K]   dWg = dG^T x, dWu = dU^T x [F][K]   (of the rounded dG and dU; bf16)
 *   dw_gate, dw_up: both, or both NULL (frozen weights; x may then be NULL)
 */
enum { LORA_ACT_SILU = 0, LORA_ACT_GELU = 1 };
enum { LORA_KEEP_NONE = 0, LORA_KEEP_BF16 = 1, LORA_KEEP_PACKED8 = 2 };
lora_status lora_gated_ffn_fwd(const void *x, const void *w_gate, const void *w_up, const float *delta_gate,
                               const float *delta_up, int act, int64_t M, int64_t K, int64_t F, void *h, int keep,
                               void *gate, void *up, void *gate_scales, void *up_scales, void *stream);
lora_status lora_gated_ffn_bwd(const void *dh, const void *x, const void *w_gate, const void *w_up, int keep,
                               const void *gate, const void *up, const void *gate_scales, const void *up_scales,
                               int act, int64_t M, int64_t K, int64_t F, void *dx, void *dgate, void *dup,
                               void *dw_gate, void *dw_up, void *stream);

/* ------------------------------------------------------------------ status
 * The tensor-core kernels of these operators bound every wait. One that runs out ends its kernel
 * early and leaves a code, (site << 8) | 1, in the library's status block of the device (the
 * first code stays): the outputs of that call, and of calls since, are then not to be used.
 *   lora_mlp_device_status        waits for the device (every stream of it); *code = the block's
 *                                 code, 0 when no kernel reported a problem. Returns LORA_OK, or
 *                                 LORA_ERR_TIMEOUT.
 *   lora_mlp_device_status_reset  waits for the device and clears the code. For tests: stall_kind
 *                                 != 0 makes the producer of that kind of kernel wait for what
 *                                 never comes; wait_limit_us != 0 sets the waits' limit.
 */
lora_status lora_mlp_device_status(int *code);
lora_status lora_mlp_device_status_reset(int stall_kind, int wait_limit_us);

#ifdef __cplusplus
}
#endif
#endif
