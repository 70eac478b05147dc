/*
 * zq_train.h -- C ABI of libzq, continued: the two ends of the data-parallel
 * step around the communication of zq.h.
 *
 *   - embedding lookup with scaling, from a table or straight from the qwZ
 *     int8 codes that the weight all-gather delivered, and the table's
 *     gradient summed by sorted tokens into the buffer that the EF quantizer
 *     or the stochastic-rounding accumulation works on;
 *   - the global norm of many gradient tensors, and clipping by it, between
 *     the reduction of the gradients and the optimizer.
 *
 * The conventions of zq.h hold (device pointers on the current device, work
 * only enqueued on `stream`, nothing allocated or kept, validation on the
 * host before anything is enqueued, 16-byte aligned data streams, 64-bit
 * indexing, calls recordable in a HIP graph), with these additions:
 *   - Device memory that a call needs for itself is a caller's `workspace`
 *     (16-byte aligned; its size comes from the host helper beside the call;
 *     its contents need no initialisation and mean nothing afterwards).  Two
 *     calls that may run at the same time, on two streams or in two graphs,
 *     need a workspace each.
 *   - Token ids are int32 or int64.  An id outside [0, rows) names no row: a
 *     lookup gives it a row of zeros and the gradient leaves the token out,
 *     so padding may carry any such id (-1, say).
 *   - Inputs may hold infinities and NaN; results follow from the formulas.
 * zq_abi_version() counts the calls of zq.h alone; a program that loads the
 * library at run time looks up the names below to see whether it has them.
 */
#ifndef ZQ_TRAIN_H
#define ZQ_TRAIN_H

#include "zq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of token ids. */
typedef enum { ZQ_I32 = 0, ZQ_I64 = 1 } zq_index_type;

/* What zq_embed_grad does with the gradient buffer. */
typedef enum {
    ZQ_GRAD_WRITE = 0,  /* writes the whole buffer                          */
    ZQ_GRAD_ADD = 1,    /* adds into it, rounded to nearest even            */
    ZQ_GRAD_ADD_SR = 2  /* adds into it, rounded stochastically (bf16 only) */
} zq_grad_mode;

/*
 * zq_embed_lookup -- embedding rows times a scale:
 *   out[t, j] = fl(scale * table[ids[t], j])  rounded to out_dtype,
 * +0 where ids[t] is outside [0, rows).
 *
 *   table  [rows, dim] fp32, bf16 or fp16 (table_dtype), read only.
 *   ids    [n_tok] int32 or int64 (id_type), aligned to their size, read only.
 *   out    [n_tok, dim] fp32, bf16 or fp16 (out_dtype), written.
 * One binary32 product per element (16-bit tables widen exactly), rounded to
 * nearest even for a 16-bit out_dtype; bit-exact.
 * Errors: ZQ_ERR_DTYPE (either dtype, id_type); ZQ_ERR_SIZE (rows == 0 or
 * dim == 0, rows above 2^31 - 2, dim above 2^31 - 1, n_tok above 2^30,
 * rows * dim or n_tok * dim above 2^60); then n_tok == 0 is a no-op;
 * ZQ_ERR_NULL; ZQ_ERR_ALIGN; ZQ_ERR_ALIAS (out overlapping table or ids).
 */
zq_status zq_embed_lookup(const void *table, zq_dtype table_dtype, uint64_t rows, uint64_t dim,
                          const void *ids, zq_index_type id_type, size_t n_tok, float scale,
                          void *out, zq_dtype out_dtype, void *stream);

/*
 * zq_embed_lookup_int8 -- the same from a table in qwZ's form (zq_quant_int8
 * over the flat rows * dim elements, any block), so that only the rows the
 * batch names are dequantized:
 *   out[t, j] = fl(scale * fl(k * s)),  e = ids[t] * dim + j,
 *   k = codes[e], s = scales[e / block],  rounded to out_dtype.
 *
 *   codes  [rows * dim] int8, scales [ceil(rows * dim / block)] fp32, read only.
 * Equal, bit for bit, to zq_dequant_int8 of the whole table into fp32 followed
 * by zq_embed_lookup.  Errors as there, and ZQ_ERR_BLOCK.
 */
zq_status zq_embed_lookup_int8(const int8_t *codes, const float *scales, uint32_t block,
                               uint64_t rows, uint64_t dim, const void *ids, zq_index_type id_type,
                               size_t n_tok, float scale, void *out, zq_dtype out_dtype,
                               void *stream);

/*
 * zq_embed_grad -- the lookup's gradient, summed by sorted tokens:
 *   S[v, j] = sum of dout[t, j] over the tokens t with ids[t] == v
 *   G[v, j] = fl(scale * S[v, j])
 *   ZQ_GRAD_WRITE:   grad[v, j] = G[v, j] rounded to grad_dtype, +0 in rows
 *                    that no token names (the whole buffer is written);
 *   ZQ_GRAD_ADD:     grad[v, j] = fl(grad[v, j] + G[v, j]) rounded to
 *                    grad_dtype, in the rows that tokens name; the other rows
 *                    are neither read nor written;
 *   ZQ_GRAD_ADD_SR:  the same rounded as zq_sr_accumulate rounds, with
 *                    element v * dim + j at index counter_base + v * dim + j
 *                    of the random stream of `seed` (bf16 only).  The seed is
 *                    part of the call, so a graph replays the same numbers.
 * The sum runs in binary32 over the tokens in ascending t, in groups whose
 * borders depend on the ids, n_tok and dim alone: equal inputs give equal bits.
 * No atomic operation touches a sum.  In a row that m tokens name, no value
 * passes through more than min(m - 1, 70 + m / 64) additions, so S is off by at
 * most that many times 2^-24 times the sum of |dout| (to first order).
 *
 *   dout   [n_tok, dim] fp32, bf16 or fp16 (d_dtype), read only.
 *   ids    [n_tok] int32 or int64 (id_type), aligned to their size, read only.
 *   grad   [rows, dim] fp32, bf16 or fp16 (grad_dtype).
 *   workspace  at least zq_embed_grad_workspace(n_tok, rows, dim) bytes.
 * Errors: ZQ_ERR_DTYPE (a dtype, id_type or mode; ZQ_GRAD_ADD_SR with another
 * grad_dtype than bf16); ZQ_ERR_SIZE (the limits of zq_embed_lookup, a
 * workspace too small, counter_base + rows * dim above 2^64 - 1);
 * ZQ_ERR_NULL; ZQ_ERR_ALIGN; ZQ_ERR_ALIAS (grad or workspace overlapping
 * another buffer).  With n_tok == 0, ZQ_GRAD_WRITE clears grad and the other
 * modes do nothing; dout, ids and workspace are not looked at.
 */
zq_status zq_embed_grad(const void *dout, zq_dtype d_dtype, const void *ids, zq_index_type id_type,
                        size_t n_tok, uint64_t rows, uint64_t dim, float scale, void *grad,
                        zq_dtype grad_dtype, zq_grad_mode mode, uint64_t seed,
                        uint64_t counter_base, void *workspace, size_t workspace_bytes,
                        void *stream);

/* Bytes of workspace zq_embed_grad needs; 0 for sizes that it refuses and for
 * n_tok == 0.  Host only. */
size_t zq_embed_grad_workspace(size_t n_tok, uint64_t rows, uint64_t dim);

/* One tensor of a gradient norm or clip: g [n] is read; zq_grad_clip_batched
 * writes out [n], which is g itself or overlaps no other range (unused, and
 * may be NULL, in zq_grad_sumsq_batched). */
typedef struct {
    const void *g;
    void *out;
    uint64_t n;
} zq_grad_segment;

/*
 * zq_grad_sumsq_batched -- the sum of squares over many gradient tensors,
 *   *sumsq = [*sumsq +] sum over all tensors and elements of x * x,
 * in binary64 throughout (a square of a binary32 value is exact there and
 * neither overflows nor vanishes), in an order fixed by the segments' sizes:
 * equal inputs give equal bits.  The relative error is at most 2^-53 times
 * the longest chain of additions: below 2^-39 up to 2^33 elements.
 *
 * The caller adds the ranks' sums (one scalar all-reduce) before the clip;
 * with accumulate != 0 a second list (another dtype, say) adds to the first.
 *   segs       HOST array of n_seg segments (read during the call only).
 *   sumsq      one binary64, 8-byte aligned, written (with accumulate != 0
 *              read first).  Written also when there is nothing to sum.
 *   workspace  at least zq_grad_sumsq_workspace(n_seg) bytes.
 * Errors: ZQ_ERR_DTYPE; ZQ_ERR_NULL (segs NULL with n_seg > 0, g of a
 * non-empty segment, sumsq, workspace); ZQ_ERR_SIZE (n_seg above 65536,
 * more than 2^40 elements together, a workspace too small); ZQ_ERR_ALIGN;
 * ZQ_ERR_ALIAS (sumsq or workspace overlapping a tensor or each other;
 * tensors may overlap each other).
 */
zq_status zq_grad_sumsq_batched(const zq_grad_segment *segs, uint32_t n_seg, zq_dtype g_dtype,
                                int accumulate, double *sumsq, void *workspace,
                                size_t workspace_bytes, void *stream);

/* Bytes of workspace zq_grad_sumsq_batched needs; 0 when n_seg is above 65536.
 * Host only. */
size_t zq_grad_sumsq_workspace(uint32_t n_seg);

/*
 * zq_grad_clip_batched -- clipping by the global norm:
 *   norm = sqrt(*sumsq);  c = min(1, max_norm / (norm + eps))   (binary64,
 *   c rounded once to binary32);  out_i = fl(c * g_i) rounded to g_dtype.
 * A NaN in *sumsq gives c = NaN, as does 0 / 0 (max_norm, eps and the norm all
 * 0); an infinity gives c = 0.  Where c == 1 and out is g itself, the tensor is
 * neither read nor written.
 *
 *   segs   HOST array of n_seg segments (read during the call only).
 *   sumsq  one binary64 on the device, read only.
 *   max_norm, eps   finite, >= 0 (ZQ_ERR_SIZE otherwise).
 *   norm   one fp32, written with the norm rounded to binary32, or NULL.
 * Errors: ZQ_ERR_DTYPE; ZQ_ERR_NULL (segs, sumsq, g or out of a non-empty
 * segment); ZQ_ERR_SIZE (also as above); ZQ_ERR_ALIGN; ZQ_ERR_ALIAS (a written range -- out,
 * norm -- overlapping any other range, except out == g of the same segment).
 */
zq_status zq_grad_clip_batched(const zq_grad_segment *segs, uint32_t n_seg, zq_dtype g_dtype,
                               const double *sumsq, float max_norm, float eps, float *norm,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZQ_TRAIN_H */
