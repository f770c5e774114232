/*
 * moe_dense.h -- C ABI of the dense operators beside the routed experts: a
 * shared expert that every token passes, and the update of the weight matrices.
 *
 *   y = layer(n) + scale * shared(n)        moe_gated_ffn, moe_gated_ffn_backward
 *   w <- w - lr * orthogonal factor of w's momentum       moe_muon_step
 *
 * Conventions as in moe.h: device pointers owned by the caller, 16-byte
 * aligned unless a call says otherwise (a NULL that a call allows is aligned),
 * asynchronous on `stream`, no allocation, no host synchronisation, argument
 * errors returned before anything is enqueued, deterministic (no floating-point
 * atomics: the same inputs give the same bits on the same device).  A workspace
 * belongs to one call at a time: calls that may run at the same time, and
 * captured graphs that may, have one each.  Its first word is a device status
 * word (moe_read_device_error), which the caller clears once before the first call;
 * the rest needs no initialisation.
 */
#ifndef MOE_GB300_DENSE_H
#define MOE_GB300_DENSE_H

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------- gated feed-forward (dense) -- */

/* The gate's activation. */
typedef enum {
    MOE_ACT_SILU = 0, /* g * sigmoid(g) */
    MOE_ACT_GELU = 1, /* the tanh form: g * sigmoid(2 sqrt(2 / pi) (g + 0.044715 g^3)) */
    MOE_ACT_RELU = 2  /* max(g, 0) */
} moe_act;

/* Bytes of workspace of the two calls (0 if a size is invalid).  Each may be
 * called with any workspace of at least its own size. */
size_t moe_gated_ffn_workspace_bytes(int32_t T, int32_t d, int32_t h);
size_t moe_gated_ffn_backward_workspace_bytes(int32_t T, int32_t d, int32_t h);

/*
 * moe_gated_ffn -- for T tokens of width d, with h hidden units:
 *   G = x Wg^T,  U = x Wu^T                        [T, h]
 *   h_act = bf16(act(G) * U)
 *   y[t]  = bf16(add[t] + token_scale[t] * (h_act[t] Wd^T))
 * and, for the backward, the two factors that it multiplies by:
 *   p_save = bf16(act(G)),  q_save = bf16(U * act'(G))     (relu'(0) = 0)
 * Products and activations are fp32; h_act, p_save, q_save and y are each
 * rounded once.  The tensor core cuts an fp32 sum, towards zero, by up to 2^-23 of its
 * size for every 16 products: terms of one sign lose up to 2^-16 at widths of 2048, 2^-11
 * at 65536 (R of the backward too), where half a step of bf16 is up to 2^-8.
 *   x [T, d], w_gate, w_up [h, d], w_down [d, h] bf16; add [T, d] bf16 or NULL
 *   (0), may be y itself; token_scale [T] fp32 or NULL (1); y out [T, d] bf16;
 *   h_act out [T, h] bf16; p_save, q_save out [T, h] bf16, both or neither NULL.
 * x is not y.  d and h are multiples of 8 and at most 65536, T at most 2^24;
 * T = 0 does nothing.
 */
moe_status moe_gated_ffn(int32_t T, int32_t d, int32_t h, int32_t act, const moe_bf16 *x,
                         const moe_bf16 *w_gate, const moe_bf16 *w_up, const moe_bf16 *w_down,
                         const moe_bf16 *add, const float *token_scale, moe_bf16 *y,
                         moe_bf16 *h_act, moe_bf16 *p_save, moe_bf16 *q_save, void *ws,
                         size_t ws_bytes, cudaStream_t stream);

/*
 * moe_gated_ffn_backward -- with s = token_scale and R = dy Wd (fp32):
 *   dU = bf16(s R p_save),  dG = bf16(s R q_save)
 *   dx           = dx_in + dG Wg + dU Wu
 *   dw_gate      = dG^T x,  dw_up = dU^T x,  dw_down = dy^T bf16(s h_act)
 *   dtoken_scale = sum over the hidden units of R * h_act
 *   x, w_*, token_scale, h_act, p_save, q_save: of the forward; dy [T, d] bf16;
 *   dx_in [T, d] of dx_dtype or NULL (0); dx out [T, d] of dx_dtype, may be
 *   dx_in itself but not x or dy; dw_gate, dw_up out [h, d], dw_down out [d, h],
 *   dtoken_scale out [T], all of dw_dtype (moe_dtype); dtoken_scale may be NULL and
 *   needs token_scale.
 * fp32 sums, each output rounded once (what is below fp32 in an fp32 output is
 * the rounding of h_act, p_save, q_save, dG, dU and, with a token scale, s h_act to
 * bf16; a sum of dx and of the weights' gradients is cut by up to 2^-14 of its size,
 * however many tokens it runs over).  The gradient of add is
 * dy.  T = 0 writes zeros to the weights' gradients.
 */
moe_status moe_gated_ffn_backward(int32_t T, int32_t d, int32_t h, const moe_bf16 *x,
                                  const moe_bf16 *w_gate, const moe_bf16 *w_up,
                                  const moe_bf16 *w_down, const float *token_scale,
                                  const moe_bf16 *h_act, const moe_bf16 *p_save,
                                  const moe_bf16 *q_save, const moe_bf16 *dy, int32_t dx_dtype,
                                  const void *dx_in, void *dx, int32_t dw_dtype, void *dw_gate,
                                  void *dw_up, void *dw_down, void *dtoken_scale, void *ws,
                                  size_t ws_bytes, cudaStream_t stream);

/* ----------------------------------------------------------- Newton-Schulz -- */

#define MOE_NS_MAX_STEPS 16

/* Bytes of workspace of moe_newton_schulz and moe_muon_step (0 if a size is
 * invalid): the iterates of all B matrices, about 4 B (2 m n + 2 m^2) bytes with m
 * the short and n the long side; the status word alone up to 128 x 256. */
size_t moe_newton_schulz_workspace_bytes(int32_t B, int32_t rows, int32_t cols);

/*
 * moe_newton_schulz -- for each of B matrices M [rows, cols], X of the shape
 * [m, n] with m <= n (M, or its transpose where rows > cols):
 *   X = M / (|M|_F + eps)
 *   steps times, with the step's (a, b, c):  S = X X^T;  X = (a I + b S + c S^2) X
 *   out = X, transposed back
 * With coefficients that lift every singular value towards 1 this is M with its
 * singular values set to about 1: the orthogonal factor of M.
 *   x [B, rows, cols] of x_dtype; out [B, rows, cols] of out_dtype, may be x
 *   itself where the types are one; both aligned to their element only;
 *   coefficients: steps x 3 floats on the host (read before the call returns), or
 *   NULL for (3.4445, -4.7750, 2.0315) in each; 1 <= steps <= MOE_NS_MAX_STEPS.
 * Precision: the iterates are held as two fp16 pieces (22 bits and more) and a
 * product is three products of pieces with fp32 sums, because a rounding error
 * grows by up to a^steps where M's singular values are small.  The pieces
 * are scaled by 2^10, which needs X's singular values below 8 throughout:
 * coefficients that can take a singular value in [0, 1] past 7.5, or the factor
 * a + b s^2 + c s^4 past 60, are refused (MOE_ERR_UNSUPPORTED).  A matrix with an
 * infinity or a NaN gives NaNs, in its own entries only.
 * |M|_F is right for entries of any size, however small or large their squares.  An
 * entry of X is held to 2^-22 of itself or to 2^-35, whichever is more, so a matrix far
 * below eps, whose X is about M / eps, keeps fewer bits than one above it.
 * rows and cols are at most 65536, eps is finite and >= 1e-30.  B = 0 does nothing.
 */
moe_status moe_newton_schulz(int32_t B, int32_t rows, int32_t cols, int32_t x_dtype, const void *x,
                             int32_t out_dtype, void *out, int32_t steps,
                             const float *coefficients, float eps, void *ws, size_t ws_bytes,
                             cudaStream_t stream);

/*
 * moe_muon_step -- one update of B weight matrices [rows, cols], in place:
 *   momentum = mu * momentum + grad
 *   u        = nesterov ? grad + mu * momentum : momentum
 *   w        = (1 - lr * weight_decay) * w - lr * scale * newton_schulz(u)
 *   w_copy   = bf16(w)
 *   w, momentum [B, rows, cols] fp32, in and out; grad [B, rows, cols] fp32; w_copy
 *   out [B, rows, cols] bf16 or NULL; lr [1] fp32 on the device (a captured step
 *   replays with the value that is there then).  The tensors are aligned to their
 *   element only, and none is another's.
 * steps, coefficients, eps and ws as in moe_newton_schulz; mu, weight_decay and
 * scale are finite.
 */
moe_status moe_muon_step(int32_t B, int32_t rows, int32_t cols, float *w, moe_bf16 *w_copy,
                         float *momentum, const float *grad, const float *lr, float mu,
                         float weight_decay, float scale, int32_t nesterov, int32_t steps,
                         const float *coefficients, float eps, void *ws, size_t ws_bytes,
                         cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_DENSE_H */
