/*
 * quads_head.h -- C ABI of the output head and of the losses on it, MI355X
 * (gfx950), in libquads.so beside the calls of quads.h.
 *
 * The method (arXiv 2607.15810) brings the rollout's and the learner's token
 * log-probabilities together (section 3, Table 3).  These calls are the two
 * ends of that comparison:
 *  - the learner's arithmetic at the rollout's shapes: bf16 activations times
 *    the NVFP4 weights that quads_nvfp4_weight_qdq writes (W4A16, Eq. (12)),
 *    for a few rows per weight matrix (a decode step's head or experts);
 *  - log-probabilities of given tokens with the entropy and the top
 *    alternatives, from logits, and their gradient;
 *  - a distillation loss from another model's top alternatives, and its
 *    gradient.
 *
 * The conventions of quads.h hold: device pointers, 16-byte aligned, dense and
 * row-major unless a row stride is stated, bf16 as uint16_t bit patterns
 * (arrays of int32 and fp32 words other than logits and outputs of a product
 * need 4-byte alignment only), asynchronous on `stream` (a stream of the calling thread's current device),
 * caller-owned workspace, host-side argument checks before any launch,
 * QUADS_* status codes, size-0 inputs a no-op.  Every call may be captured
 * into a HIP graph.  Results do not depend on the order in which work-groups
 * run: the same inputs give the same bits.
 *
 * Logits.  z [T, V], `dtype` QUADS_OUT_F32 or QUADS_OUT_BF16, row t at element
 * t * ld (ld >= V; elements V .. ld - 1 of a row are neither read nor
 * written).  1 <= V < 2^30, T < 2^24, ld < 2^31.  0 < inv_temp <= 1e30, it below;
 * probabilities are those of softmax(it * z).  Entries may be -inf (masked):
 * their probability is 0.  A row whose every entry is -inf has entropy 0, the
 * stats (-inf, 0) and a zero gradient.  A row with +inf or NaN gives NaN.
 *   stats  fp32 [T, 2]: (m, s), m = max_v z_v, s = ln sum_v exp(it (z_v - m)),
 *          so that ln p_v = it (z_v - m) - s; kept as two numbers, since
 *          their sum in fp32 would lose what the backward pass needs
 */
#ifndef QUADS_HEAD_H
#define QUADS_HEAD_H

#include "quads.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of alternatives per row. */
#define QUADS_TOP_MAX 128

/*
 * W4A16 grouped product for few rows per expert (Eq. (12) in the forward
 * direction, on the NVFP4 codes themselves): for packed row p of expert e,
 *   Y[p, n] = s_tW[e] sum_{j<K} x[row(p), j] w_e[n, j],   w the exact v*s_b.
 *   x          bf16 [Tx, K], finite, K % 16 == 0, K < 2^26; rows < 2^24
 *   row_token  NULL: row(p) = p (Tx = rows); else int32 [rows], row(p) =
 *              row_token[p] < Tx
 *   w_nib, w_scale, w_ts, offsets, E, N, epilogue, out_dtype, out   as in
 *              quads_moe_w4a4_gemm (offsets may be NULL when E == 1)
 * Any number of rows is computed, with one read of an expert's weights per 16
 * or 32 of its rows: larger batches belong to a GEMM.
 * The error is below (176 + K / 512) 2^-24 sum |x w| per output element plus
 * the rounding to bf16, and 2^-28 times the largest |x| of a row's 512-channel
 * block times sum |w| where a block spans more than 28 binary orders.
 * Workspace: none (quads_moe_w4a16_gemv_ws is 0 for every size, ws is not used).
 */
size_t quads_moe_w4a16_gemv_ws(int64_t rows, int64_t K, int32_t E, int64_t N);
int quads_moe_w4a16_gemv(const uint16_t* x, const int32_t* row_token, int64_t rows, int64_t K,
                         const uint8_t* w_nib, const uint8_t* w_scale, const float* w_ts,
                         const int32_t* offsets, int32_t E, int64_t N, int epilogue,
                         int out_dtype, void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * Log-probabilities of given tokens, entropy and top alternatives.
 *   ids       int32 [T]: the token of each row; a value outside [0, V) means
 *             none, and logp[t] = 0.  NULL (with logp NULL): no tokens
 *   topk      0 <= topk <= min(V, QUADS_TOP_MAX)
 *   logp      out fp32 [T]: ln p of the token (-inf where its entry is -inf)
 *   entropy   NULL or out fp32 [T]: -sum_v p_v ln p_v
 *   stats     out fp32 [T, 2]
 *   top_logp, top_id   out fp32, int32 [T, topk] (NULL when topk == 0): the
 *             topk largest entries of the row, descending, equal entries in
 *             ascending index order.  In a row with +inf or NaN, top_id
 *             holds distinct indices in [0, V) in no stated order.
 */
size_t quads_token_logprob_ws(int64_t T, int64_t V, int32_t topk);
int quads_token_logprob(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                        const int32_t* ids, float inv_temp, int32_t topk, float* logp,
                        float* entropy, float* stats, float* top_logp, int32_t* top_id,
                        void* ws, size_t ws_bytes, void* stream);

/*
 * Gradient of quads_token_logprob's logp and entropy H:
 *   dz_v = it (g_logp (1[v = id] - p_v) - g_entropy p_v (ln p_v + H))
 *   stats, entropy    the forward call's (entropy may be NULL when g_entropy is)
 *   g_logp, g_entropy NULL (no such gradient) or fp32 [T]; g_logp of a row
 *             without a token is ignored
 *   dlogits   out [T, V] in the logits' type and row stride; may be logits
 */
int quads_token_logprob_backward(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                 const int32_t* ids, float inv_temp, const float* stats,
                                 const float* entropy, const float* g_logp,
                                 const float* g_entropy, void* dlogits, void* stream);

/*
 * Distillation from another model's top alternatives:
 *   loss[t] = w_t sum_i q_i (ln q_i - ln p_{id_i})
 *   t_val, t_id   fp32, int32 [T, topk], 1 <= topk <= QUADS_TOP_MAX; entries
 *             whose id is outside [0, V) are left out; an id may stand more
 *             than once in a row
 *   renorm    1: q = softmax(it * t_val) over the row's entries (t_val are
 *             logits or log-probabilities at temperature 1);
 *             0: q = exp(t_val) (t_val are log-probabilities at the loss's
 *             temperature; their sum may stay below 1)
 *   weight    NULL (1) or fp32 [T]; a row of weight 0 has loss and gradient 0
 *             and its logits are not read
 *   loss      out fp32 [T] (an entry with q > 0 and p = 0 gives +inf)
 *   stats     out fp32 [T, 2] of the logits ((0, 0) for a row of weight 0)
 * quads_topk_distill_backward: dz_v = g_t w_t it (Q p_v - q_v), Q = sum_i q_i,
 * q_v the sum over the entries with id v; g fp32 [T]; dlogits as in
 * quads_token_logprob_backward.
 * quads_topk_distill_grad: loss and dlogits (g = 1) in one call; dlogits may
 * be logits.
 */
size_t quads_topk_distill_ws(int64_t T, int64_t V, int32_t topk);
int quads_topk_distill(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                       const float* t_val, const int32_t* t_id, int32_t topk,
                       const float* weight, float inv_temp, int renorm, float* loss,
                       float* stats, void* ws, size_t ws_bytes, void* stream);
int quads_topk_distill_backward(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                const float* t_val, const int32_t* t_id, int32_t topk,
                                const float* weight, float inv_temp, int renorm,
                                const float* stats, const float* g, void* dlogits, void* stream);
size_t quads_topk_distill_grad_ws(int64_t T, int64_t V, int32_t topk);
int quads_topk_distill_grad(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                            const float* t_val, const int32_t* t_id, int32_t topk,
                            const float* weight, float inv_temp, int renorm, float* loss,
                            void* dlogits, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QUADS_HEAD_H */
