/*
 * quads_block.h -- C ABI of the layer around the experts, MI355X (gfx950), in
 * libquads.so beside the calls of quads.h.
 *
 * What stands between the residual stream and the grouped products of quads.h
 * (arXiv 2607.15810, section 3: an MoE layer of the rollout and of the learner):
 *  - the residual's addition with the root-mean-square norm, whose output
 *    enters the quantizers (bf16 with partial maxima of its magnitude) or the
 *    MX product (FP8 codes and scales), and its gradient;
 *  - the router's top experts with their weights, and their gradient;
 *  - the learner's tokens in expert order and back, with the routing weights
 *    applied, and the gradients (the rollout's products gather by row_token
 *    and need no sorted copy).
 *
 * The conventions of quads.h hold: device pointers, 16-byte aligned (arrays of
 * int32 and fp32 words other than rows of channels: 4-byte), dense and
 * row-major unless a row stride is stated, bf16 as uint16_t bit patterns,
 * asynchronous on `stream` (a stream of the calling thread's current device),
 * caller-owned workspace, host-side argument checks before any launch, QUADS_*
 * status codes, size-0 inputs a no-op.  Types are QUADS_OUT_F32 or
 * QUADS_OUT_BF16.  A row stride is in elements, at least the row's length and
 * below 2^31; elements between the rows are neither read nor written.  Every
 * call may be captured into a HIP graph.  The same inputs give the same bits:
 * no result depends on the order in which work-groups run.  Inputs need not be
 * finite: a NaN or an infinity shows in the rows (and weights' gradients) that
 * it enters, as the formulas give it, and in no others.
 */
#ifndef QUADS_BLOCK_H
#define QUADS_BLOCK_H

#include "quads.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Output type of quads_rmsnorm: the codes of quads_mx_quantize (QUADS_MX_FP8). */
#define QUADS_OUT_MX_FP8 2

/*
 * Residual addition and root-mean-square norm of T rows of H channels:
 *   h = x + residual, formed in fp32 and rounded to the residual's type
 *       (h = x without a residual)
 *   y = h / sqrt(mean_j h_j^2 + eps) * weight
 *   x, ldx, x_dtype                rows of x
 *   residual, ldr, res_dtype       NULL or the rows of the residual stream
 *   weight, w_dtype                NULL (ones) or [H]
 *   eps                            1e-70 <= eps <= 1e70
 *   sum        NULL or out [T, H] in the residual's type: h (NULL without a
 *              residual).  May be residual, or x, where that is dense and of
 *              the residual's type
 *   y, out_dtype   out [T, H]: fp32, bf16, or QUADS_OUT_MX_FP8: E4M3 codes
 *              uint8 with a scale byte per 32 channels in `scales` [T, H/32]
 *              (H % 32 == 0), the format and rules of quads_mx_quantize applied
 *              to y itself, not to its bf16 rounding; a NaN gets a NaN code, an
 *              infinite y saturates, and their block has the scale byte 254, the
 *              largest (quads_mx_quantize asks for finite input).  y may be x or
 *              residual, where that is dense and of y's type and not sum
 *   amax_part  NULL, or (bf16 only) out uint32 [amax_groups]: partial maxima of
 *              |y| as bf16 bits for quads_nvfp4_quantize_partials and
 *              quads_rac_quantize_partials; amax_groups >=
 *              quads_rmsnorm_amax_groups(T, H), the rest is written 0
 * 1 <= H < 2^24, T < 2^31.  The mean is formed in fp64; with QUADS_OUT_MX_FP8
 * so is y (each code and scale is that of the exact y unless it lies within
 * about 2^-50 of a border).  fp32 and bf16 outputs come from two fp32 products
 * (3 * 2^-24 of the value, and 2^-149 (|weight| + 1) where h / sqrt(..) or y is
 * subnormal; two bits more in rows whose root mean square is above 2^126) and
 * are rounded once.
 */
int64_t quads_rmsnorm_amax_groups(int64_t T, int64_t H);
int quads_rmsnorm(const void* x, int x_dtype, int64_t T, int64_t H, int64_t ldx,
                  const void* residual, int res_dtype, int64_t ldr, const void* weight,
                  int w_dtype, double eps, void* sum, void* y, int out_dtype, uint8_t* scales,
                  uint32_t* amax_part, int64_t amax_groups, void* stream);

/*
 * Gradient of quads_rmsnorm's fp32 or bf16 output y and of h.  With n = h r,
 * r = 1 / sqrt(mean h^2 + eps), c = mean_j n_j w_j g_j:
 *   dh = g_sum + r (w g - n c),   dweight_j = sum_t g_tj n_tj
 *   g, g_dtype     [T, H]: the gradient of y
 *   h, h_dtype, ldh    the call's h: its sum, or x where there was no residual
 *   g_sum      NULL (0) or [T, H] in h's type: the gradient that h gets elsewhere
 *   dx, dx_dtype   out [T, H]: dh in x's type.  May be g, or g_sum, of that type
 *   dres       NULL or out [T, H]: dh in h's type, for a residual of another
 *              type than x.  Not dx; may be g_sum
 *   dweight    NULL or out [H] in w_dtype (a NULL weight has none)
 * Sums over channels are fp64; the sum over tokens is fp32 in chains of at most
 * 64 + 127 additions (rows, then parts of a work-group) joined in fp64, in an
 * order that the sizes alone decide.
 * ws: quads_rmsnorm_backward_ws bytes (0 without dweight for rows that one
 * work-group holds).
 */
size_t quads_rmsnorm_backward_ws(int64_t T, int64_t H, int want_dweight);
int quads_rmsnorm_backward(const void* g, int g_dtype, const void* h, int h_dtype, int64_t T,
                           int64_t H, int64_t ldh, const void* weight, int w_dtype, double eps,
                           const void* g_sum, void* dx, int dx_dtype, void* dres, void* dweight,
                           void* ws, size_t ws_bytes, void* stream);

/*
 * Routing: the topk experts with the largest logits of each token, and their
 * weights, from p = softmax(z) over the E experts.
 *   logits     z [T, E], `dtype`, row stride ld; 1 <= E <= 4096, T < 2^24
 *   topk       1 <= topk <= min(E, 64)
 *   renorm     0: w_i = p_{id_i};  1: divided by their sum over the token's
 *              topk (the softmax over the chosen logits)
 *   topk_ids   out int32 [T, topk]: descending by logit, equal logits (0 and
 *              -0 among them) in ascending index order; quads_moe_pack's input
 *   topk_w     out fp32 [T, topk]
 * A logit of -inf masks an expert: its weight is 0 (it is named, in index
 * order, only where fewer than topk others are left).  In a token with every
 * logit -inf every weight is 0; with +inf or NaN the weights are NaN (or 0)
 * and the ids distinct and in [0, E).
 * Weights are formed in fp32: numerators exp(z - max z) by expf, the terms of the
 * sum over all experts (renorm 0) by 2^x of a rounded product, each off by up to
 * 2.5 * 2^-24 |z - max z| of itself.
 */
int quads_moe_route(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, int32_t topk,
                    int renorm, int32_t* topk_ids, float* topk_w, void* stream);

/*
 * Gradient of quads_moe_route's weights, with a_i = g_i w_i, A = sum_i a_i:
 *   renorm 0: dz_v = (a_i where v = id_i) - p_v A
 *   renorm 1: dz_v = a_i - w_i A where v = id_i, 0 elsewhere
 *   topk_ids, topk_w   the forward call's;  g fp32 [T, topk]
 *   logits     the forward call's (may be NULL with renorm 1)
 *   dlogits    out [T, E] in `dtype`, dense; may be logits where ld == E
 * A token with every logit -inf has gradient 0.  An id outside [0, E) is left
 * out of both sums.  The exponential in p_v is off by the rounding of z_v - max z
 * in fp32 and 2 ulps, however unlikely the expert (0 below 2^-126).
 */
int quads_moe_route_backward(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld,
                             const int32_t* topk_ids, const float* topk_w, const float* g,
                             int32_t topk, int renorm, void* dlogits, void* stream);

/*
 * Tokens in packed (expert) order: out[pos[t * topk + s]] = x[t] for every
 * token t and slot s.  pos is quads_moe_pack's, or any other placement.
 *   x          [T, H], `dtype`, row stride ldx; 1 <= H < 2^24, T < 2^24,
 *              1 <= topk <= 64, T * topk < 2^31
 *   pos        int32 [T * topk]: a value outside [0, rows) means that the slot
 *              is left out.  A row is named once at most (named more often, each
 *              of its channels is one of its slots', any of them)
 *   out        [rows, H], 0 <= rows < 2^31; not x
 *   zero_rest  0: rows of out that no slot names are left as they were;  1: they
 *              are zeroed, with quads_moe_sort_ws bytes of workspace (4 a row for
 *              large outputs, else 0; its content is of no account)
 */
size_t quads_moe_sort_ws(int64_t rows, int64_t H, int dtype, int zero_rest);
int quads_moe_sort(const void* x, int dtype, int64_t T, int64_t H, int64_t ldx,
                   const int32_t* pos, int32_t topk, int64_t rows, int zero_rest, void* out,
                   void* ws, size_t ws_bytes, void* stream);

/*
 * Back into token order: out[t] = sum over slots in order of
 * topk_w[t, s] * y[pos[t * topk + s]], accumulated in fp32 and rounded once;
 * slots that are left out add nothing (and their weight is not used).
 *   y          [rows, H], y_dtype;  pos, T, topk, H, rows as in quads_moe_sort
 *   topk_w     NULL (ones: the gradient of quads_moe_sort) or fp32 [T, topk]
 *   out        [T, H], out_dtype; not y
 */
int quads_moe_unsort(const void* y, int y_dtype, int64_t rows, const int32_t* pos,
                     const float* topk_w, int64_t T, int32_t topk, int64_t H, void* out,
                     int out_dtype, void* stream);

/*
 * Gradient of quads_moe_unsort, for a pos that names a row once at most:
 *   dy[pos[t * topk + s]] = topk_w[t, s] g[t];  dw[t, s] = sum_j g_tj y[pos, j]
 *   g          [T, H], g_dtype
 *   y, y_dtype the forward call's (may be NULL when dw is)
 *   dy         NULL or out [rows, H] in y's type; may be y (zero_rest 0)
 *   zero_rest, ws   rows of dy that no slot names, as in quads_moe_sort (the
 *              workspace for y's type)
 *   dw         NULL or out fp32 [T, topk], summed in fp32; 0 where the slot is
 *              left out.  NULL when topk_w is
 */
int quads_moe_unsort_backward(const void* g, int g_dtype, const void* y, int y_dtype,
                              int64_t rows, const int32_t* pos, const float* topk_w, int64_t T,
                              int32_t topk, int64_t H, int zero_rest, void* dy, float* dw,
                              void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QUADS_BLOCK_H */
