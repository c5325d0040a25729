// Gradient of the residual addition with the norm (formulas in norm.h).
#include "norm.h"

namespace quads {
namespace norm {

// ---------------------------------------------------------------- gradient --
struct GradArgs {
    const void* g;
    const void* h;
    const void* weight;
    const void* g_sum;
    void* dx;
    void* dres;
    float2* stat;                            // [T]: r, c
    float* part;                             // [runs, H], with dweight
    int64_t T, H, ldh;
    int64_t rows;                            // of a run of rows
    int runs;
    double eps, inv_h;
    int w_dtype, dx_dtype;
};
constexpr int kThreads = 256;
// (r, c) of each row.
template <int kG, int kH>
__global__ __launch_bounds__(kThreads) void k_rms_grad_stat(GradArgs a) {
    __shared__ double s_part[2][kMaxWaves];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void* g = row_at<kG>(a.g, t * a.H);
        const void* h = row_at<kH>(a.h, t * a.ldh);
        double sq = 0.0, dot = 0.0;
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
            const Raw<kG> gr = load<kG>(g, c, a.H - c);
            const Raw<kH> hr = load<kH>(h, c, a.H - c);
            float w[kPer];
            load_weight(a.weight, a.w_dtype, c, a.H - c, w);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const double hd = hr.get(i);
                sq = fma(hd, hd, sq);
                dot = fma(hd, (double)(gr.get(i) * w[i]), dot);
            }
        }
        const double rd = rsqrt(group_sum(sq, s_part, 0) * a.inv_h + a.eps);
        const double c = group_sum(dot, s_part, 1) * a.inv_h * rd;
        if (threadIdx.x == 0) a.stat[t] = make_float2((float)rd, (float)c);
    }
}

// dh, and the weight gradient's partial sums, of eight channels a thread in the
// rows of run blockIdx.y.  Each value of g and g_sum is read before its place is
// written, by the same thread.
template <int kG, int kH>
__global__ __launch_bounds__(kThreads) void k_rms_grad_apply(GradArgs a) {
    const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kPer;
    if (c >= a.H) return;
    const int64_t n = a.H - c, t0 = blockIdx.y * a.rows;
    const int64_t t1 = t0 + a.rows < a.T ? t0 + a.rows : a.T;
    float w[kPer], acc[kPer] = {};
    load_weight(a.weight, a.w_dtype, c, n, w);
    for (int64_t t = t0; t < t1; ++t) {
        const Raw<kG> gr = load<kG>(row_at<kG>(a.g, t * a.H), c, n);
        const Raw<kH> hr = load<kH>(row_at<kH>(a.h, t * a.ldh), c, n);
        const float2 st = a.stat[t];
        float d[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float nm = hr.get(i) * st.x;
            acc[i] = fmaf(gr.get(i), nm, acc[i]);
            d[i] = st.x * fmaf(-st.y, nm, gr.get(i) * w[i]);
        }
        if (a.g_sum) {
            const Raw<kH> s = load<kH>(row_at<kH>(a.g_sum, t * a.H), c, n);
#pragma unroll
            for (int i = 0; i < kPer; ++i) d[i] += s.get(i);
        }
        if (a.dres) store<kH>(row_at<kH>(a.dres, t * a.H), c, n, pack<kH>(d));
        if (a.dx_dtype == QUADS_OUT_BF16)
            store<1>(row_at<1>(a.dx, t * a.H), c, n, pack<1>(d));
        else
            store<0>(row_at<0>(a.dx, t * a.H), c, n, pack<0>(d));
    }
    if (a.part) store<0>(a.part + blockIdx.y * a.H, c, n, pack<0>(acc));
}

__global__ __launch_bounds__(kThreads) void k_rms_join_weight(const float* part, int groups,
                                                              int64_t H, void* dweight, int bf16) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= H) return;
    double s = 0.0;
    for (int i = 0; i < groups; ++i) s += (double)part[i * H + c];
    if (bf16) ((uint16_t*)dweight)[c] = (uint16_t)bf16_bits((float)s, 0.0f);
    else ((float*)dweight)[c] = (float)s;
}

constexpr int64_t kMaxGroups = 2048;
inline int64_t row_groups(int64_t T) { return T < kMaxGroups ? T : kMaxGroups; }
// Runs of rows: one weight gradient's partial sum each.
inline int64_t grad_runs(int64_t T) { return T < 8 ? 1 : (T / 8 < 512 ? T / 8 : 512); }

template <int kG, int kH>
void launch_grad(const GradArgs& a, hipStream_t s) {
    const dim3 block(kThreads);
    hipLaunchKernelGGL((k_rms_grad_stat<kG, kH>), dim3((unsigned)row_groups(a.T)), block, 0, s, a);
    const unsigned cols = (unsigned)((a.H + kThreads * kPer - 1) / (kThreads * kPer));
    hipLaunchKernelGGL((k_rms_grad_apply<kG, kH>), dim3(cols, (unsigned)a.runs), block, 0, s, a);
}

}  // namespace norm
}  // namespace quads

using namespace quads;

extern "C" size_t quads_rmsnorm_backward_ws(int64_t T, int64_t H, int want_dweight) {
    if (norm::check_sizes(T, H, H) != QUADS_OK || T == 0) return 0;
    return align_up((size_t)T * 8, 256) +
           (want_dweight ? align_up((size_t)norm::grad_runs(T) * H * 4, 256) : 0);
}

extern "C" int quads_rmsnorm_backward(const void* g, int g_dtype, const void* h, int h_dtype,
                                      int64_t T, int64_t H, int64_t ldh, const void* weight,
                                      int w_dtype, double eps, const void* g_sum, void* dx,
                                      int dx_dtype, void* dres, void* dweight, void* ws,
                                      size_t ws_bytes, void* stream) {
    using namespace norm;
    if (int e = check_sizes(T, H, ldh)) return e;
    if (!ok_type(g_dtype) || !ok_type(h_dtype) || !ok_type(dx_dtype) ||
        (weight && !ok_type(w_dtype)))
        return QUADS_EINVAL;
    if (!ok_eps(eps)) return QUADS_EINVAL;
    if ((dweight && (!weight || !ok_ptr(dweight))) || !ok_opt_ptr(weight)) return QUADS_EINVAL;
    hipStream_t s = (hipStream_t)stream;
    const int w_bf16 = w_dtype == QUADS_OUT_BF16;
    const dim3 join((unsigned)((H + kThreads - 1) / kThreads));
    if (T == 0) {                            // no rows: their sum is 0
        if (dweight) {
            hipLaunchKernelGGL(k_rms_join_weight, join, dim3(kThreads), 0, s, nullptr, 0, H, dweight,
                               w_bf16);
            QUADS_CHECK_LAUNCH();
        }
        return QUADS_OK;
    }
    if (!ok_ptr(g) || !ok_ptr(h) || !ok_opt_ptr(g_sum) || !ok_ptr(dx) || !ok_opt_ptr(dres) ||
        dres == dx || dx == h || (dx == g && dx_dtype != g_dtype) ||
        (dx == g_sum && dx_dtype != h_dtype) || (dres && (dres == h || dres == g)))
        return QUADS_EINVAL;
    const size_t need = quads_rmsnorm_backward_ws(T, H, dweight != nullptr);
    if (need && (ws_bytes < need || !ok_ptr(ws))) return QUADS_EWORKSPACE;
    const int64_t runs = grad_runs(T);
    float* part = dweight ? (float*)((char*)ws + align_up((size_t)T * 8, 256)) : nullptr;
    GradArgs a = {g, h, weight, g_sum, dx, dres, (float2*)ws, part, T, H, ldh,
                  (T + runs - 1) / runs, (int)runs, eps, 1.0 / (double)H, weight ? w_dtype : kNoWeight,
                  dx_dtype};
    const bool gb = g_dtype == QUADS_OUT_BF16, hb = h_dtype == QUADS_OUT_BF16;
    if (gb && hb) launch_grad<1, 1>(a, s);
    else if (gb) launch_grad<1, 0>(a, s);
    else if (hb) launch_grad<0, 1>(a, s);
    else launch_grad<0, 0>(a, s);
    QUADS_CHECK_LAUNCH();
    if (dweight) {
        hipLaunchKernelGGL(k_rms_join_weight, join, dim3(kThreads), 0, s, a.part, (int)runs, H,
                           dweight, w_bf16);
        QUADS_CHECK_LAUNCH();
    }
    return QUADS_OK;
}
