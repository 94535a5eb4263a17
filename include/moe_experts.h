/*
 * moe_experts.h -- C ABI of the operators around the experts, in the same
 * library as moe_ep.h (libmoe_ep.so, one AMD Instinct MI355X, gfx950): the
 * router in front of the layout, the experts' FP8 products and activation
 * between dispatch and combine, and the gradients of router, activation and
 * combine.
 *
 * One layer, forward:
 *   moe_gate -> topk_idx, topk_weights
 *   moe_layout_dispatch / moe_ll_layout_dispatch_fp8 / moe_dispatch_fp8 -> FP8 rows
 *   moe_grouped_gemm_fp8 (gate and up columns) -> moe_swiglu_fp8
 *   moe_grouped_gemm_fp8 (down) -> moe_combine
 * and backward: moe_combine_grad (rows and weights), moe_swiglu_grad,
 * moe_combine with topk_weights = NULL (the gradient of the dispatch is the
 * plain sum of a token's rows), moe_gate_grad. The gradient of a product with
 * respect to its rows is the product of the cast gradient (moe_quantize_fp8) with
 * the transposed weights; the gradient with respect to the weights is not part
 * of this library.
 *
 * The conventions of moe_ep.h hold: caller-owned device pointers, nothing
 * allocated, freed or kept between calls, every call enqueues on the caller's
 * stream without waiting, MOE_OK or a negative MOE_ERR_* code before anything
 * is enqueued, data errors OR-ed into an optional device status word. Every
 * call may be captured into a HIP graph, and calls on several streams share
 * nothing. The caller's current device is the one the pointers live on.
 *
 * Segments. The calls on expert rows take row_start [E] and count [E] (int32,
 * device): expert e's rows are row_start[e] ... row_start[e] + count[e] - 1 of
 * a buffer of `rows` rows. A layout's offset and count arrays are just that,
 * for the contiguous and for the low-latency layout. Rows of no segment are
 * neither read nor written. A segment that does not lie in [0, rows) is
 * skipped and sets MOE_STATUS_BAD_SLOT; count <= 0 means no rows. Segments
 * must not overlap.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Router options. */
#define MOE_GATE_BF16 1    /* logits (and d_logits) are bf16, else float */
#define MOE_GATE_SIGMOID 2 /* scores are sigmoid(logit), else softmax over the E experts */
#define MOE_GATE_RENORM 4  /* the selected scores are divided by their sum */

#define MOE_STATUS_BAD_LOGIT 16 /* a NaN or +infinity among the logits: never selected */

/* Router: the K best experts of each token and their weights.
 *   logits [T*E] float or bf16. Larger logit first, equal logits by lower id.
 *   -infinity masks an expert: it is never selected, and a token with fewer
 *   than K unmasked experts gets id -1 and weight 0 in its last places (which
 *   the layouts and the combine skip). NaN and +infinity are treated as
 *   -infinity and set MOE_STATUS_BAD_LOGIT. The lowest finite value is an
 *   ordinary logit.
 *   topk_idx [T*K] int64, topk_weights [T*K] float:
 *     softmax:           w_k = scale * exp(x_k) / sum over all e of exp(x_e)
 *     softmax + renorm:  w_k = scale * exp(x_k) / sum over the selected j of exp(x_j)
 *     sigmoid:           w_k = scale / (1 + exp(-x_k))
 *     sigmoid + renorm:  w_k = scale * s_k / sum over the selected j of s_j
 *   (the renormalised sigmoids from log s, so that sums which would underflow
 *   do not divide by zero).
 * 0 <= T <= 2^26 - 64, 1 <= E <= 1024, 1 <= K <= min(E, 64), scale finite. logits and topk_weights
 * 4-byte aligned (bf16 logits: 2), topk_idx 8-byte. status may be NULL. */
int moe_gate(int32_t T, int32_t E, int32_t K, const void *logits, int64_t *topk_idx,
             float *topk_weights, int32_t flags, float scale, int32_t *status,
             hipStream_t stream);

/* Gradient of moe_gate's weights with respect to the logits, the selection
 * held fixed: d_logits [T*E] (the logits' type; every entry is written) from
 * d_weights [T*K] float, the logits and ids of the forward call, and the same
 * flags and scale. An id of -1 or on a masked logit contributes nothing, and
 * masked logits get 0; an id outside [-1, E) sets MOE_STATUS_BAD_EXPERT and
 * is skipped. */
int moe_gate_grad(int32_t T, int32_t E, int32_t K, const void *logits, const int64_t *topk_idx,
                  const float *d_weights, void *d_logits, int32_t flags, float scale,
                  int32_t *status, hipStream_t stream);

/* Gradient of moe_combine / moe_combine_masked: for every pair (t,k) with a
 * slot,
 *   d_y[slot] = bf16_rne( w[t*K+k] * d_out[t] )      (one float product)
 *   d_weights[t*K+k] = sum over h of d_out[t][h] * y[slot][h], in float,
 * and d_weights = 0 for a pair without one. topk_weights NULL: all ones.
 * d_weights NULL: not computed, and y is not read (it may be NULL). With
 * rank_mask [R] (and topk_idx [T*K], both or neither), a pair on a masked rank
 * took no part in the sum: its row of d_y is +0 and its weight's gradient 0.
 *   Rows of d_y that no pair maps to are left untouched. Each row belongs to
 *   one pair, as the layouts write them: the same slot twice is not supported
 *   (one of the two products is left in the row). A slot outside
 *   [-1, recv_rows) sets MOE_STATUS_BAD_SLOT (also on a masked rank: its row
 *   would be written), gets d_weights 0 and no row.
 * Needs (T + 7) * K <= 2^24 - 16 and the shape limits of moe_combine. d_out, y
 * and d_y 16-byte aligned, d_y must not overlap d_out or y. The gradient of the
 * dispatch is moe_combine with topk_weights = NULL. */
int moe_combine_grad(const moe_shape *shape, const uint16_t *d_out, const uint16_t *y,
                     int64_t recv_rows, const int32_t *slot, const float *topk_weights,
                     uint16_t *d_y, float *d_weights, const int64_t *topk_idx,
                     const int32_t *rank_mask, int32_t *status, hipStream_t stream);

/* Each expert's product on FP8 rows: for every row r of expert e's segment and
 * 0 <= n < N,
 *   out[r][n] = bf16_rne( sum over g of a_scale(r, g) * w_scale[e][n / 128][g]
 *                         * sum over c in group g of a[r][c] * w[e][n][c] )
 * with groups of 128 channels, summed in float.
 *   a [rows*C] E4M3 codes and their scales as the FP8 dispatch calls and
 *   moe_quantize_fp8 write them: flags has MOE_FP8_SCALE_ROWS for row-major
 *   scales ([rows][C/128] float, or [rows][C/512] words with MOE_FP8_UE8M0);
 *   without it they are column-major in each expert's rows/E rows
 *   ([E][C/128][rows/E], rows % E == 0, segment e within rows
 *   [e*rows/E, (e+1)*rows/E), else MOE_STATUS_BAD_SLOT), the format of the
 *   low-latency dispatch. MOE_FP8_ROUND_SCALE is accepted and changes nothing.
 *   w [E*N*C] E4M3 codes, row-major in C; w_scale [E][ceil(N/128)][C/128] float.
 *   out [rows*N] bf16; rows of no segment are left untouched.
 *   max_count: no segment holds more rows than this (a low-latency batch's T or
 *   M), 0 if unknown. It lets a small batch run as one launch; a segment with
 *   more rows is skipped and sets MOE_STATUS_BAD_SLOT.
 * C % 128 == 0 (512 with UE8M0), N % 8 == 0, 8 <= N, C <= 2^20, E <= 1024.
 * a, w and out 16-byte aligned, scales 4-byte aligned. A row's scale times a
 * block's must be a finite float (the two are multiplied first; below 2^-126 the
 * product loses bits). The gradient with respect to the rows is the same call on
 * d_out, cast by moe_quantize_fp8, and on weights stored transposed: w [E*C*N],
 * w_scale with its blocks changed over. N is the channel count there, so it
 * takes N % 128 == 0 (512 with UE8M0); for another N both are stored with N
 * rounded up, the added channels 0. */
int moe_grouped_gemm_fp8(int32_t E, int32_t N, int32_t C, const uint8_t *a, const void *a_scale,
                         int64_t rows, const int32_t *row_start, const int32_t *count,
                         const uint8_t *w, const float *w_scale, uint16_t *out, int32_t flags,
                         int32_t max_count, int32_t *status, hipStream_t stream);

/* The activation between an expert's two products, cast to FP8: for every row
 * of a segment, with g = x[r][0..I) and u = x[r][I..2I),
 *   h = g / (1 + exp(-g)) * u   (float, kept within the finite floats; 0 where
 *                                exp(-g) passes them)
 * cast as moe_quantize_fp8 casts a row (flags as there): q [rows*I] codes,
 * scale [rows][I/128] float or [rows][I/512] words, row-major. x [rows*2I]
 * bf16; a NaN or infinity in it gives its group of 128 channels the scale NaN
 * (UE8M0: byte 255) and NaN codes, so that it shows in every result of its row's
 * product, and touches no other group. I % 128 == 0 (512 with MOE_FP8_UE8M0). x
 * and q 16-byte aligned, scale 4-byte. */
int moe_swiglu_fp8(int32_t E, int32_t I, int64_t rows, const uint16_t *x,
                   const int32_t *row_start, const int32_t *count, uint8_t *q, void *scale,
                   int32_t flags, int32_t *status, hipStream_t stream);

/* Gradient of the activation (the cast passes the gradient through): for every
 * row of a segment, with s = 1 / (1 + exp(-g)),
 *   d_x[r][0..I)  = bf16_rne( d_h * u * s * (1 + g * (1 - s)) )
 *   d_x[r][I..2I) = bf16_rne( d_h * g * s )
 * x [rows*2I], d_h [rows*I], d_x [rows*2I] bf16, 16-byte aligned;
 * d_x may be x itself. NaN and infinities go as the formulas take them, each to
 * its own channel. I % 8 == 0, I <= 2^20. */
int moe_swiglu_grad(int32_t E, int32_t I, int64_t rows, const uint16_t *x, const uint16_t *d_h,
                    const int32_t *row_start, const int32_t *count, uint16_t *d_x,
                    int32_t *status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
