// Distillation from another model's top alternatives and its gradient
// (include/quads_head.h).
#include "logits.h"

namespace quads {
namespace head {

struct Rows {
    const void* z;
    int64_t T, V, ld;
    float it;
};

template <int kBf16>
__device__ __forceinline__ float ld_z(const void* z, int64_t i) {
    return kBf16 ? bf16_to_f32(((const uint16_t*)z)[i]) : ((const float*)z)[i];
}
template <int kBf16>
__device__ __forceinline__ void st_z(void* z, int64_t i, float v) {
    if (kBf16) ((uint16_t*)z)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else ((float*)z)[i] = v;
}

// Reductions over the work-group; s_red holds one value per thread.
__device__ __forceinline__ float group_max(float v, float* s_red) {
    __syncthreads();
    s_red[threadIdx.x] = v;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o) {
            const float b = s_red[threadIdx.x + o], a = s_red[threadIdx.x];
            s_red[threadIdx.x] = (a != a || a > b) ? a : b;      // NaN stays
        }
        __syncthreads();
    }
    return s_red[0];
}
__device__ __forceinline__ float group_sum(float v, float* s_red) {
    __syncthreads();
    s_red[threadIdx.x] = v;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o) s_red[threadIdx.x] += s_red[threadIdx.x + o];
        __syncthreads();
    }
    return s_red[0];
}

// m = max z, s = sum exp(it (z - m)), u = sum exp(d) d with d = it (z - m);
// (-inf, 1, 0) for a row without an unmasked entry.
template <int kBf16>
__device__ __forceinline__ void row_stats(const Rows& r, int64_t t, float* s_red, float* m_out,
                                          float* s_out, float* u_out) {
    const int64_t b = t * r.ld;
    float m = -INFINITY;
    for (int64_t v = threadIdx.x; v < r.V; v += kThreads) {
        const float z = ld_z<kBf16>(r.z, b + v);
        m = (z != z || z > m) ? z : m;
    }
    m = group_max(m, s_red);
    if (m == -INFINITY) {
        *m_out = m; *s_out = 1.0f; *u_out = 0.0f;
        return;
    }
    float s = 0.0f, u = 0.0f;
    for (int64_t v = threadIdx.x; v < r.V; v += kThreads) {
        const float d = (ld_z<kBf16>(r.z, b + v) - m) * r.it;
        const float e = expf(d);
        s += e;
        u += e * fmaxf(d, -200.0f);
    }
    *m_out = m;
    *s_out = group_sum(s, s_red);
    *u_out = group_sum(u, s_red);
}

// The teacher's distribution over its list, in LDS: s_q[i] = q_i (0 for an
// entry left out), returns Q = sum q; s_lq[i] = ln q_i.
__device__ __forceinline__ float teacher(const float* val, const int32_t* id, int topk, int64_t V,
                                         float it, int renorm, float* s_q, float* s_lq,
                                         float* s_red) {
    const int i = threadIdx.x;
    const bool have = i < topk && id[i] >= 0 && id[i] < V;
    float y = have ? (renorm ? it * val[i] : val[i]) : -INFINITY;
    if (renorm) {
        const float m = group_max(y, s_red);
        const float s = group_sum(y == -INFINITY ? 0.0f : expf(y - m), s_red);
        y = y == -INFINITY ? y : y - m - logf(s);
    }
    const float q = expf(y);
    if (i < topk) { s_q[i] = q; s_lq[i] = y; }
    return group_sum(q, s_red);
}

// mode bits: 1 = loss and stats from the logits, 2 = gradient
template <int kBf16, int kMode>
__global__ __launch_bounds__(kThreads) void k_topk_distill(Rows r, const float* t_val,
                                                           const int32_t* t_id, int topk,
                                                           const float* weight, int renorm,
                                                           float* loss, float* stats,
                                                           const float* stats_in, const float* g,
                                                           void* dz) {
    __shared__ float s_red[kThreads], s_q[QUADS_TOP_MAX], s_lq[QUADS_TOP_MAX];
    const int64_t t = blockIdx.x;
    const float w = weight ? weight[t] : 1.0f;
    if (w == 0.0f) {
        if ((kMode & 1) && threadIdx.x == 0) {
            loss[t] = 0.0f;
            if (stats) stats[2 * t] = stats[2 * t + 1] = 0.0f;
        }
        if (kMode & 2)
            for (int64_t v = threadIdx.x; v < r.V; v += kThreads) st_z<kBf16>(dz, t * r.ld + v, 0.0f);
        return;
    }
    t_val += t * topk;
    t_id += t * topk;
    const float q_all = teacher(t_val, t_id, topk, r.V, r.it, renorm, s_q, s_lq, s_red);
    float m, ls;
    if (kMode & 1) {
        float s, u;
        row_stats<kBf16>(r, t, s_red, &m, &s, &u);
        ls = logf(s);
        float y = 0.0f;
        const int i = threadIdx.x;
        if (i < topk && s_q[i] > 0.0f) {
            const float z = ld_z<kBf16>(r.z, t * r.ld + t_id[i]);
            y = s_q[i] * (s_lq[i] - (z == -INFINITY && m == m ? z : (z - m) * r.it - ls));
        }
        y = group_sum(y, s_red);
        if (threadIdx.x == 0) {
            loss[t] = w * y;
            if (stats) { stats[2 * t] = m; stats[2 * t + 1] = ls; }
        }
    } else {
        m = stats_in[2 * t];
        ls = stats_in[2 * t + 1];
    }
    if (kMode & 2) {
        const float by = w * r.it * (g ? g[t] : 1.0f);
        __syncthreads();
        for (int64_t v = threadIdx.x; v < r.V; v += kThreads) {
            float p = 0.0f;
            if (m != -INFINITY) {
                p = q_all * expf((ld_z<kBf16>(r.z, t * r.ld + v) - m) * r.it - ls);
                for (int i = 0; i < topk; ++i) p -= t_id[i] == v ? s_q[i] : 0.0f;
            }
            st_z<kBf16>(dz, t * r.ld + v, by * p);
        }
    }
}

int check_list(int64_t T, const float* t_val, const int32_t* t_id, int32_t topk,
               const float* weight, int renorm) {
    if (topk < 1 || topk > QUADS_TOP_MAX) return QUADS_ESHAPE;
    if (renorm != 0 && renorm != 1) return QUADS_EINVAL;
    if (T == 0) return QUADS_OK;
    return ok_ptr4(t_val) && ok_ptr4(t_id) && ok_opt4(weight) ? QUADS_OK : QUADS_EINVAL;
}

}  // namespace head
}  // namespace quads

using namespace quads;

extern "C" size_t quads_topk_distill_ws(int64_t T, int64_t V, int32_t topk) {
    (void)T; (void)V; (void)topk;
    return 0;
}

#define QUADS_DISTILL(MODE, ...)                                                               \
    do {                                                                                       \
        const head::Rows r{logits, T, V, ld, inv_temp};                                        \
        const dim3 grid((unsigned)T), block(head::kThreads);                                   \
        hipStream_t st = (hipStream_t)stream;                                                  \
        if (dtype == QUADS_OUT_BF16)                                                           \
            hipLaunchKernelGGL((head::k_topk_distill<1, MODE>), grid, block, 0, st, r, t_val,  \
                               t_id, (int)topk, weight, renorm, __VA_ARGS__);                  \
        else                                                                                   \
            hipLaunchKernelGGL((head::k_topk_distill<0, MODE>), grid, block, 0, st, r, t_val,  \
                               t_id, (int)topk, weight, renorm, __VA_ARGS__);                  \
        QUADS_CHECK_LAUNCH();                                                                  \
        return QUADS_OK;                                                                       \
    } while (0)

extern "C" int quads_topk_distill(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                  const float* t_val, const int32_t* t_id, int32_t topk,
                                  const float* weight, float inv_temp, int renorm, float* loss,
                                  float* stats, void* ws, size_t ws_bytes, void* stream) {
    int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc == QUADS_OK) rc = head::check_list(T, t_val, t_id, topk, weight, renorm);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!ok_ptr4(loss) || !ok_ptr4(stats)) return QUADS_EINVAL;
    const size_t need = quads_topk_distill_ws(T, V, topk);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return QUADS_EWORKSPACE;
    QUADS_DISTILL(1, loss, stats, (const float*)nullptr, (const float*)nullptr, (void*)nullptr);
}

extern "C" int quads_topk_distill_backward(const void* logits, int dtype, int64_t T, int64_t V,
                                           int64_t ld, const float* t_val, const int32_t* t_id,
                                           int32_t topk, const float* weight, float inv_temp,
                                           int renorm, const float* stats, const float* g,
                                           void* dlogits, void* stream) {
    int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc == QUADS_OK) rc = head::check_list(T, t_val, t_id, topk, weight, renorm);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!ok_ptr4(stats) || !ok_ptr4(g) || !ok_ptr(dlogits)) return QUADS_EINVAL;
    QUADS_DISTILL(2, (float*)nullptr, (float*)nullptr, stats, g, dlogits);
}

extern "C" int quads_topk_distill_grad(const void* logits, int dtype, int64_t T, int64_t V,
                                       int64_t ld, const float* t_val, const int32_t* t_id,
                                       int32_t topk, const float* weight, float inv_temp,
                                       int renorm, float* loss, void* dlogits, void* ws,
                                       size_t ws_bytes, void* stream) {
    int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc == QUADS_OK) rc = head::check_list(T, t_val, t_id, topk, weight, renorm);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!ok_ptr4(loss) || !ok_ptr(dlogits)) return QUADS_EINVAL;
    const size_t need = quads_topk_distill_ws(T, V, topk);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return QUADS_EWORKSPACE;
    QUADS_DISTILL(3, loss, (float*)nullptr, (const float*)nullptr, (const float*)nullptr, dlogits);
}
