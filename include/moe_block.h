/*
 * moe_block.h -- C ABI of the operators that surround the routed-expert layer
 * in a pre-norm training block:
 *
 *   h_i = h_{i-1} + y_{i-1};  n_i = layer_norm(h_i);  y_i = layer(n_i)
 *   loss = task loss + a * balance_i + b * z_i
 *
 *   - layer norm, fused with the residual add, and its backward with the
 *     reduction of the weight's gradient;
 *   - the router's balance loss and z loss over per-expert counts, their
 *     gradient with respect to every logit, and the dense router gradient
 *     that carries it to the tokens and the router weight;
 *   - activation checkpoints of the experts' saved buffers in 8 bits, and the
 *     backward steps that read them.
 * The pages behind moe.h describe none of these; each call states its own
 * definition.
 *
 * Conventions as in moe.h: device pointers owned by the caller, 16-byte
 * aligned (a NULL that a call allows is aligned), asynchronous on `stream`,
 * no allocation, no host synchronisation, argument errors returned before
 * anything is enqueued, deterministic (no floating-point atomics: the same
 * inputs give the same bits on the same device).
 */
#ifndef MOE_GB300_BLOCK_H
#define MOE_GB300_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors that a call takes in more than one type. */
typedef enum {
    MOE_BF16 = 0,
    MOE_FP32 = 1
} moe_dtype;

/* ------------------------------------------------------------ layer norm -- */

/*
 * moe_layer_norm -- residual add and layer norm of `rows` rows of width d:
 *   s[t]    = x[t] + add[t]     (rounded to x's type and written to x_sum;
 *                                s = x when add is NULL)
 *   mean[t] = sum_j s[t, j] / d
 *   rstd[t] = 1 / sqrt(sum_j (s[t, j] - mean[t])^2 / d + eps)
 *   y[t, j] = bf16((s[t, j] - mean[t]) * rstd[t] * gamma[j] + beta[j])
 * in fp32, the variance from the centred values (a large mean does not cancel
 * in it).  The norm is taken of the rounded sum, which is what the
 * backward reads.
 *   x [rows, d] of x_dtype; add [rows, d] bf16 or NULL; gamma, beta [d] fp32,
 *   each may be NULL (1 and 0); x_sum out [rows, d] of x_dtype, required with
 *   add, NULL without it, may be x itself; y out [rows, d] bf16; mean, rstd out
 *   [rows] fp32 (kept for the backward), both or neither NULL.
 * eps must be finite and > 0; d a multiple of 8, at most 16384
 * (MOE_ERR_UNSUPPORTED above).  rows = 0 does nothing.
 */
moe_status moe_layer_norm(int32_t rows, int32_t d, int32_t x_dtype, const void *x,
                          const moe_bf16 *add, const float *gamma, const float *beta, float eps,
                          void *x_sum, moe_bf16 *y, float *mean, float *rstd, cudaStream_t stream);

/* Bytes of workspace moe_layer_norm_backward needs (per-CTA partial sums of
 * the weight gradients; 0 if rows or d is invalid). */
size_t moe_layer_norm_backward_workspace_bytes(int32_t rows, int32_t d);

/*
 * moe_layer_norm_backward -- with xh = (x - mean) * rstd and w = dy * gamma:
 *   dx[t, j]  = dres[t, j] + rstd[t] * (w[t, j] - sum_i w[t, i] / d
 *                                       - xh[t, j] * sum_i w[t, i] xh[t, i] / d)
 *   dgamma[j] = sum_t dy[t, j] * xh[t, j];   dbeta[j] = sum_t dy[t, j]
 *   x [rows, d] of x_dtype: the normalised rows (x_sum of the forward, or its
 *   x without add); dy [rows, d] of dy_dtype; gamma [d] fp32 or NULL (1);
 *   mean, rstd [rows] fp32 from the forward; dres [rows, d] of dx_dtype or NULL
 *   (0): the gradient that reaches the residual stream past the norm; dx out
 *   [rows, d] of dx_dtype, may be dres itself; dgamma, dbeta out [d] fp32,
 *   each may be NULL; ws of moe_layer_norm_backward_workspace_bytes bytes,
 *   256-byte aligned.
 * fp32 throughout, dx rounded once.  Each column of dgamma and dbeta is summed
 * in a fixed order.  rows = 0 writes zeros to dgamma and dbeta.
 */
moe_status moe_layer_norm_backward(int32_t rows, int32_t d, int32_t x_dtype, const void *x,
                                   int32_t dy_dtype, const void *dy, const float *gamma,
                                   const float *mean, const float *rstd, int32_t dx_dtype,
                                   const void *dres, void *dx, float *dgamma, float *dbeta,
                                   void *ws, size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------- balance loss -- */

/* Bytes of workspace moe_balance_loss needs (per-CTA partial sums; 0 if the
 * shape is invalid). */
size_t moe_balance_loss_workspace_bytes(const moe_shape *s);

/*
 * moe_balance_loss -- how evenly the router spreads the tokens.  A token t
 * counts if token_mask is NULL or token_mask[t] != 0 (0 marks padding); Tc
 * tokens count.
 *   p[t]            = softmax(logits[t])           over all N experts
 *   lse[t]          = log sum_e exp(logits[t, e])  (0 for a token that does not count)
 *   expert_count[e] = routes (t, k) of counted tokens with topk_idx = e
 *   expert_prob[e]  = sum over counted t of p[t, e] / Tc
 *   losses[0]       = N * sum_e expert_count[e] / (Tc * K) * expert_prob[e]
 *                     (1 when both are even)
 *   losses[1]       = sum over counted t of lse[t]^2 / Tc
 * Tc = 0 gives zeros.  expert_count is moe_route's expert_demand when every
 * token counts; entries of topk_idx outside [0, N) are skipped.
 *   logits [T, N] fp32 (moe_route leaves them at moe_route_logits_offset of its
 *   workspace); topk_idx [T, K] int32; token_mask [T] uint8 or NULL;
 *   expert_count out [N] int32; token_count out [1] int32 (Tc); expert_prob
 *   out [N] fp32; lse out [T] fp32; losses out [2] fp32; ws of
 *   moe_balance_loss_workspace_bytes bytes, 256-byte aligned.
 * A logit of -inf has probability 0; a counted token whose logits are all
 * -inf has lse -inf, probabilities 0 and adds nothing to losses[1].  NaN and
 * +inf logits of counted tokens give NaN losses; the logits of other
 * tokens are not read.  Uses T, N and K of the shape.  Sums are fp32 in a fixed
 * order, counts are exact.
 */
moe_status moe_balance_loss(const moe_shape *s, const float *logits, const int32_t *topk_idx,
                            const uint8_t *token_mask, int32_t *expert_count,
                            int32_t *token_count, float *expert_prob, float *lse, float *losses,
                            void *ws, size_t ws_bytes, cudaStream_t stream);

/*
 * moe_balance_loss_backward -- the gradient with respect to every logit, the
 * counts held fixed:
 *   dlogits[t, j] = p[t, j] * (dlosses[0] * N / Tc * (f[j] - sum_e p[t, e] f[e])
 *                              + dlosses[1] * 2 / Tc * lse[t])
 *                   + sum over k with topk_idx[t, k] = j of dlogit[t, k]
 * with f[e] = expert_count[e] / (Tc * K); the first line is 0 for a token that
 * does not count.  The second line, left out when dlogit is NULL, adds the
 * gradient of the gates (moe_combine_backward_checkpoint's dlogit, or
 * moe_router_backward's), so that dlogits is the router's whole gradient; it
 * applies to every token.
 *   logits, topk_idx, token_mask as in the forward; expert_count, token_count
 *   and lse as it wrote them (or, for a loss over several batches, the sums of
 *   their counts); dlosses [2] fp32 on the device: the gradients of losses[0] and
 *   losses[1], for instance the two losses' weights; dlogit [T, K] fp32 or NULL;
 *   dlogits out [T, N] fp32, every element written.
 */
moe_status moe_balance_loss_backward(const moe_shape *s, const float *logits,
                                     const int32_t *topk_idx, const uint8_t *token_mask,
                                     const int32_t *expert_count, const int32_t *token_count,
                                     const float *lse, const float *dlosses, const float *dlogit,
                                     float *dlogits, cudaStream_t stream);

/* Bytes of workspace moe_router_dense_backward needs (0 if the shape is
 * invalid). */
size_t moe_router_dense_backward_workspace_bytes(const moe_shape *s);

/*
 * moe_router_dense_backward -- the router's products for a gradient of every
 * logit (moe_router_weight_backward takes only the K chosen ones):
 *   dx[t, :]       = dx_in[t, :] + sum_e dlogits[t, e] * w_router[e, :]
 *   dw_router[e, :] = sum_t dlogits[t, e] * x[t, :]
 *   dbias[e]       = sum_t dlogits[t, e]
 *   x [T, d] bf16; w_router [N, d] fp32; dlogits [T, N] fp32; dx_in [T, d] fp32
 *   or NULL (0), for instance moe_dispatch_backward's dx; dx out [T, d] fp32, may
 *   be dx_in itself, NULL to leave it out; dw_router out [N, d] fp32 or NULL;
 *   dbias out [N] fp32 or NULL; ws of moe_router_dense_backward_workspace_bytes
 *   bytes, 256-byte aligned, word 0 the device status word.
 * Products and sums keep fp32 accuracy: in the 2-norm about the error of a chain
 * of fp32 multiply-adds of the same length, or less.  A non-finite dlogit or
 * weight makes what it reaches non-finite, inf or NaN.  Uses T, d and N of the
 * shape.
 */
moe_status moe_router_dense_backward(const moe_shape *s, const moe_bf16 *x, const float *w_router,
                                     const float *dlogits, const float *dx_in, float *dx,
                                     float *dw_router, float *dbias, void *ws, size_t ws_bytes,
                                     cudaStream_t stream);

/* ----------------------------------------------------- 8-bit checkpoints -- */

/*
 * Activation checkpoints hold packed capacity buffers in MXINT8, the 8-bit
 * integer format of the OCP Microscaling (MX) v1.0 specification: blocks of
 * 32 consecutive elements of a row share one scale 2^E, stored as the byte
 * E + 127, E = floor(log2 max|v|) clamped below at -127 (an all-zero block
 * gets byte 0); an element is the signed byte c = v * 2^(6 - E) rounded to
 * nearest, ties to even, and held to [-127, 127]; its value is c * 2^(E - 6),
 * which bf16 holds exactly.  A block with a NaN or an infinity gets byte 255
 * and codes 0, and reads back as 32 NaNs: a broken activation is not hidden.
 * Against the E4M3 codes of moe_mxfp8.h the same byte carries 6 to 7
 * significant bits instead of 4 near the block's maximum, which is what the
 * backward's products weigh most.
 *   codes [rows, cols] int8, scales [rows, cols / 32] uint8, both row-major.
 * Only the packed rows before expert_offset[N] (read on the device) are read
 * or written.  d and h must be multiples of 32 (MOE_ERR_UNSUPPORTED).
 */

/*
 * moe_checkpoint_save -- the experts' saved buffers in 8 bits, so that one set
 * of bf16 buffers serves every layer:
 *   g_save, u_save [R, h] -> g_q, u_q [R, h], g_scale, u_scale [R, h / 32]
 *   y_disp [R, d]         -> y_q [R, d], y_scale [R, d / 32]
 *   expert_offset [N + 1] as moe_route wrote it.  A buffer whose source is
 *   NULL is left out (its outputs may then be NULL).
 */
moe_status moe_checkpoint_save(const moe_shape *s, const int32_t *expert_offset,
                               const moe_bf16 *g_save, const moe_bf16 *u_save,
                               const moe_bf16 *y_disp, int8_t *g_q, uint8_t *g_scale, int8_t *u_q,
                               uint8_t *u_scale, int8_t *y_q, uint8_t *y_scale,
                               cudaStream_t stream);

/*
 * moe_checkpoint_restore -- the operands of moe_expert_ffn_backward from the
 * checkpoint: g_save and u_save get the codes' values (exact in bf16), and
 *   h_act = bf16(silu(G) * U)   of those values, in fp32
 *   (moe_expert_ffn's h_act recomputed; it needs no checkpoint of its own).
 */
moe_status moe_checkpoint_restore(const moe_shape *s, const int32_t *expert_offset,
                                  const int8_t *g_q, const uint8_t *g_scale, const int8_t *u_q,
                                  const uint8_t *u_scale, moe_bf16 *g_save, moe_bf16 *u_save,
                                  moe_bf16 *h_act, cudaStream_t stream);

/*
 * moe_combine_backward_checkpoint -- moe_combine_backward with y_disp read from
 * its checkpoint:
 *   dy_disp[route_row[t, k]] = bf16(topk_gate[t, k] * dy[t])   (fp32 product)
 *   dgate[t, k] = <dy[t], value(y_q, y_scale)[route_row[t, k]]>  (fp32; 0 if dropped)
 * and, when dlogit is not NULL, the chosen logits' gradient through the gates'
 * softmax, as moe_router_backward defines it:
 *   dlogit[t, k] = topk_gate[t, k] * (dgate[t, k] - sum_k' topk_gate[t, k'] * dgate[t, k'])
 * (moe_balance_loss_backward takes it from here).  dgate, dlogit out [T, K] fp32.
 */
moe_status moe_combine_backward_checkpoint(const moe_shape *s, const moe_bf16 *dy,
                                           const int8_t *y_q, const uint8_t *y_scale,
                                           const int32_t *route_row, const float *topk_gate,
                                           moe_bf16 *dy_disp, float *dgate, float *dlogit,
                                           cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_BLOCK_H */
