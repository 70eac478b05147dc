/*
 * zq_layers.h -- C ABI of libzq, continued: the training step between the
 * embedding lookup and the gradient buffers, in the int8 blocks of zq.h.
 *
 *   - SwiGLU whose inputs are kept for the backward pass as int8 blocks, and
 *     its gradient from them;
 *   - a linear layer's weight gradient from its input kept as int8 blocks
 *     (zq_quant_int8 of the activation, or the codes above);
 *   - softmax cross entropy of the vocabulary projection, worked through in
 *     pieces of the vocabulary so that the logits are never kept, with its
 *     gradient; the projection as 16-bit values or as the qwZ int8 codes that the
 *     weight all-gather delivered, widened a piece at a time into the workspace.
 *
 * The conventions of zq.h and zq_train.h hold: device pointers on the current
 * device, work only enqueued on `stream`, nothing allocated or kept, validation
 * on the host before anything is enqueued, 16-byte aligned data streams (4 for
 * scales, loss, lse and dloss), a caller's `workspace` for each call that may
 * run at the same time (16-byte aligned, no initialisation, its size from the
 * host helper beside the call), calls recordable in a HIP graph.  Inputs may
 * hold infinities and NaN; results follow from the formulas.
 *
 * Matrix products take bf16 or fp16 operands and sum in binary32 in an order
 * fixed by the sizes: equal inputs give equal bits.  No sum is touched by an
 * atomic operation.  A value kept as an int8 block enters a product as
 * zq_dequant_int8 gives it in the product's type: fl(k * s) rounded to nearest
 * even.
 */
#ifndef ZQ_LAYERS_H
#define ZQ_LAYERS_H

#include "zq_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * zq_swiglu_int8 -- the gated product, with its inputs kept as int8 blocks:
 *   h[i] = gate[i] * sigmoid(gate[i]) * up[i]   rounded to dtype
 *   gate_codes, gate_scales = zq_quant_int8(gate);  up_codes, up_scales likewise
 * in one pass over the inputs.  Codes and scales equal zq_quant_int8's bit for
 * bit.  h is formed in binary32 from the inputs themselves (not from the kept
 * values), off by at most 2^-21 times itself before its rounding (a sigmoid below
 * 2^-126 counts as 0).
 *
 *   gate, up   [n] fp32, bf16 or fp16 (dtype), read only; they may be one buffer.
 *   h          [n] of dtype, written.
 *   *_codes    [n] int8, *_scales [ceil(n / block)] fp32, written.
 * As for zq_quant_int8, a NaN or infinity makes its own block's scale and codes
 * meaningless; h is unaffected elsewhere.
 * Errors: ZQ_ERR_DTYPE, ZQ_ERR_BLOCK, ZQ_ERR_SIZE (n above 2^60); then n == 0 is
 * a no-op; ZQ_ERR_NULL; ZQ_ERR_ALIGN; ZQ_ERR_ALIAS (an output overlapping
 * another buffer).
 */
zq_status zq_swiglu_int8(const void *gate, const void *up, zq_dtype dtype, size_t n, uint32_t block,
                         void *h, int8_t *gate_codes, float *gate_scales, int8_t *up_codes,
                         float *up_scales, void *stream);

/*
 * zq_swiglu_grad_int8 -- its gradient at the kept values g = k * s (gate) and
 * u = k * s (up), with sg = sigmoid(g):
 *   dgate[i] = dh[i] * u * sg * (1 + g * (1 - sg))
 *   dup[i]   = dh[i] * g * sg
 *   h[i]     = g * sg * u          (where h is not NULL: the input of the layer
 *                                   that follows, for its weight gradient)
 * in binary32, rounded once to dtype.
 *
 *   dh              [n] of dtype, read only.
 *   dgate, dup, h   [n] of dtype, written; h may be NULL.
 * Errors as above.
 */
zq_status zq_swiglu_grad_int8(const int8_t *gate_codes, const float *gate_scales,
                              const int8_t *up_codes, const float *up_scales, uint32_t block,
                              const void *dh, zq_dtype dtype, size_t n, void *dgate, void *dup,
                              void *h, void *stream);

/*
 * zq_linear_grad_int8 -- a linear layer's weight gradient from its kept input:
 *   G[o, i] = sum over t of dy[t, o] * x[t, i],   x[t, i] = fl(k * s) rounded to
 *   dtype,  e = t * in_dim + i,  k = codes[e],  s = scales[e / block]
 *   ZQ_GRAD_WRITE: grad = G rounded to grad_dtype;
 *   ZQ_GRAD_ADD:   grad = fl(grad + G) rounded to grad_dtype.
 *
 *   dy      [n_tok, out_dim] bf16 or fp16 (dtype), read only.
 *   codes   [n_tok * in_dim] int8, scales [ceil(n_tok * in_dim / block)] fp32.
 *   grad    [out_dim, in_dim] fp32, bf16 or fp16 (grad_dtype).
 *   workspace  at least zq_linear_grad_workspace(n_tok, out_dim, in_dim) bytes.
 * Errors: ZQ_ERR_DTYPE (dtype fp32, another mode than the two); ZQ_ERR_BLOCK;
 * ZQ_ERR_SIZE (out_dim or in_dim 0 or above 2^20, their product above 2^36, n_tok
 * above 2^20, a workspace too small); ZQ_ERR_NULL; ZQ_ERR_ALIGN; ZQ_ERR_ALIAS (grad or workspace
 * overlapping another buffer).  With n_tok == 0, ZQ_GRAD_WRITE clears grad and
 * ZQ_GRAD_ADD does nothing; dy, codes, scales and workspace are not looked at.
 */
zq_status zq_linear_grad_int8(const void *dy, zq_dtype dtype, const int8_t *codes,
                              const float *scales, uint32_t block, size_t n_tok, uint64_t out_dim,
                              uint64_t in_dim, void *grad, zq_dtype grad_dtype, zq_grad_mode mode,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace zq_linear_grad_int8 needs; 0 for sizes that it refuses and
 * for n_tok == 0.  Host only. */
size_t zq_linear_grad_workspace(size_t n_tok, uint64_t out_dim, uint64_t in_dim);

/*
 * zq_ce_loss -- softmax cross entropy of the vocabulary projection, per token:
 *   z[t, v] = scale * sum over j of x[t, j] * w[v, j]
 *   lse[t]  = log of the sum over v of exp(z[t, v])
 *   loss[t] = lse[t] - z[t, ids[t]]
 * A token whose id is outside [0, rows) is left out: its loss and lse are +0 and
 * its x has no effect (padding may hold anything).
 *
 *   x      [n_tok, dim] bf16 or fp16 (dtype), read only.
 *   w      [rows, dim] of dtype, read only.
 *   ids    [n_tok] int32 or int64 (id_type), aligned to their size, read only.
 *   loss   [n_tok] fp32, written.
 *   lse    [n_tok] fp32, written: what zq_ce_grad needs.
 *   scale  any number; 0 makes all logits equal (and NaN where a sum is not finite).
 *   piece  rows of w worked on at a time (rounded up to a multiple of 256), or 0 for
 *          the library's choice: a larger piece takes a larger workspace and fewer
 *          launches.
 *   workspace  at least zq_ce_loss_workspace(n_tok, rows, dim, piece) bytes.
 * The sum runs in binary32 over tiles of the vocabulary, each with a maximum of
 * its own taken out; nothing of size n_tok * rows is stored.  The loss is formed as
 * log(1 + the sum over the other rows of exp(z[t, v] - z[t, ids[t]])), so that it is
 * never negative and its relative precision does not depend on its size: beyond what
 * the logits' sums themselves are off by, at most 2^-22 times the logits' differences
 * and 2^-23 (64 + rows / 2048) of itself.
 * Errors: ZQ_ERR_DTYPE (dtype fp32, id_type); ZQ_ERR_SIZE (rows or dim 0, rows
 * above 2^24, dim above 2^20, n_tok above 2^20, n_tok * dim above 2^36, a
 * workspace too small); then n_tok == 0 is a no-op; ZQ_ERR_NULL; ZQ_ERR_ALIGN; ZQ_ERR_ALIAS (loss, lse or
 * workspace overlapping another buffer).
 */
zq_status zq_ce_loss(const void *x, zq_dtype dtype, size_t n_tok, uint64_t dim, const void *w,
                     uint64_t rows, const void *ids, zq_index_type id_type, float scale,
                     float *loss, float *lse, uint64_t piece, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * zq_ce_loss_int8 -- the same with w in qwZ's form: codes [rows * dim] int8 and
 * scales [ceil(rows * dim / block)] fp32, as zq_quant_int8 writes them for the
 * flat matrix; w[v, j] is what zq_dequant_int8 gives in dtype, formed a piece at
 * a time.  Errors as there, and ZQ_ERR_BLOCK.
 */
zq_status zq_ce_loss_int8(const void *x, zq_dtype dtype, size_t n_tok, uint64_t dim,
                          const int8_t *codes, const float *scales, uint32_t block, uint64_t rows,
                          const void *ids, zq_index_type id_type, float scale, float *loss,
                          float *lse, uint64_t piece, void *workspace, size_t workspace_bytes,
                          void *stream);

/* Bytes of workspace the two calls above need; 0 for sizes that they refuse and
 * for n_tok == 0.  Host only. */
size_t zq_ce_loss_workspace(size_t n_tok, uint64_t rows, uint64_t dim, uint64_t piece);

/*
 * zq_ce_grad -- its gradient, for the loss's gradients dloss:
 *   q[t, v]  = dloss[t] * (exp(z[t, v] - lse[t]) - (v == ids[t] ? 1 : 0))
 *   dx[t, j] = scale * sum over v of q[t, v] * w[v, j]    rounded to dtype
 *   G[v, j]  = scale * sum over t of q[t, v] * x[t, j]
 *   ZQ_GRAD_WRITE: dw = G rounded to dw_dtype;  ZQ_GRAD_ADD: dw = fl(dw + G)
 *   rounded to dw_dtype.
 * Tokens that are left out have dx = +0 and no part in dw; their x, lse and
 * dloss are not used.  The logits are formed again, a piece of the vocabulary at a
 * time, and rounded to binary32 as for the loss; q is rounded to dtype before the two
 * products (the matrix units take 16-bit operands): an error of at most half a step of dtype per q, of the
 * size that the rounding of dx to dtype has (with 128 tokens or fewer q is kept in
 * two 16-bit parts, and the error is 2^-8 of that in bf16, 2^-11 in fp16).  It is
 * the same for an fp32 dw, whose 32 bits are for adding many micro-batches.  In fp16, q is scaled by the
 * power of two that brings the largest finite |dloss| to [2^14, 2^15) and back
 * afterwards: a q below 2^-39 times that maximum vanishes.
 *
 *   lse     [n_tok] fp32 as zq_ce_loss wrote it, read only.
 *   dloss   [n_tok] fp32, read only.
 *   dx      [n_tok, dim] of dtype, written, or NULL.
 *   dw      [rows, dim] fp32, bf16 or fp16 (dw_dtype), or NULL (not both NULL).
 *   workspace  at least zq_ce_grad_workspace(n_tok, rows, dim, piece) bytes.
 * Errors as for zq_ce_loss; ZQ_ERR_DTYPE also for dw_dtype and for another mode
 * than the two.  With n_tok == 0, ZQ_GRAD_WRITE clears dw, and nothing else is
 * looked at.
 */
zq_status zq_ce_grad(const void *x, zq_dtype dtype, size_t n_tok, uint64_t dim, const void *w,
                     uint64_t rows, const void *ids, zq_index_type id_type, float scale,
                     const float *lse, const float *dloss, void *dx, void *dw, zq_dtype dw_dtype,
                     zq_grad_mode mode, uint64_t piece, void *workspace, size_t workspace_bytes,
                     void *stream);

/* zq_ce_grad_int8 -- the same with w in qwZ's form (its gradient dw is that of
 * the dequantized values). */
zq_status zq_ce_grad_int8(const void *x, zq_dtype dtype, size_t n_tok, uint64_t dim,
                          const int8_t *codes, const float *scales, uint32_t block, uint64_t rows,
                          const void *ids, zq_index_type id_type, float scale, const float *lse,
                          const float *dloss, void *dx, void *dw, zq_dtype dw_dtype,
                          zq_grad_mode mode, uint64_t piece, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Bytes of workspace the two calls above need; 0 for sizes that they refuse and
 * for n_tok == 0.  Host only. */
size_t zq_ce_grad_workspace(size_t n_tok, uint64_t rows, uint64_t dim, uint64_t piece);

#ifdef __cplusplus
}
#endif

#endif /* ZQ_LAYERS_H */
