// Residual addition with the root-mean-square norm, and its gradient.
//
//   h = RN(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = h r w
//   n = h r,  c = mean(n w g),  dh = g_sum + r (w g - n c),  dw = sum_t g n
//
// Simple form: a work-group per row, the row read twice.  h^2 of two bf16 or
// fp32 numbers and their sum are held in fp64: the sum cannot overflow, and the
// 8-bit output's codes are decided by exact comparisons of y with the format's
// borders, which fp32 statistics would move.
#include "block.h"

namespace quads {
namespace norm {

using namespace block;

constexpr int kThreads = 256;
constexpr int kNone = 2;                     // no residual

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
// Sum over the work-group, in every thread; s_part: one per wave.
__device__ __forceinline__ double group_sum(double v, double* s_part) {
    v = wave_sum(v);
    __syncthreads();                         // the values of the sum before are read
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    for (int i = 0; i < (int)blockDim.x / 64; ++i) t += s_part[i];
    return t;
}

// A double as its upper word with the lower word's bits gathered in the lowest
// one: 20 bits of mantissa behind which nothing is lost that a rounding to three
// bits or a comparison of magnitudes could need.
__device__ __forceinline__ uint32_t upper(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return (uint32_t)(b >> 32) | ((uint32_t)b != 0u);
}
// Exponent of an MX block from the largest magnitude's upper word.
__device__ __forceinline__ int mx_exponent(uint32_t top) {
    const int e = (int)(top >> 20) - 1023 - 8;
    return e < -127 ? -127 : (e > 127 ? 127 : e);
}
// v * 2^-e for the conversion to E4M3: clamped to 448, 0 below 2^-126, NaN kept.
__device__ __forceinline__ float mx_scaled(uint32_t v, int e) {
    const uint32_t a = v & 0x7FFFFFFFu;
    int t = (int)a - ((1023 - 127 + e) << 20);
    t = t < (1 << 20) ? 0 : t;
    t = t > ((127 + 9) << 20) ? ((127 + 9) << 20) : t;
    float f = __builtin_fminf(__uint_as_float((uint32_t)t << 3), 448.0f);
    f = a > 0x7FF00000u ? __uint_as_float(0x7FC00000u) : f;
    return __uint_as_float(__float_as_uint(f) | (v & 0x80000000u));
}
__device__ __forceinline__ words2 mx_codes(const float* f) {
    words2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
        c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], r, true);
    }
    return c;
}

struct Args {
    const void* x;
    const void* residual;
    const void* weight;
    void* sum;
    void* y;
    uint8_t* scales;
    uint32_t* amax_part;
    int64_t T, H, ldx, ldr;
    int64_t amax_groups;
    double eps, inv_h;
    int w_dtype;                             // -1: no weight
};

__device__ __forceinline__ void load_weight(const Args& a, int64_t c, int64_t n, float* w) {
    if (a.w_dtype == QUADS_OUT_BF16) {
        const Raw<1> r = load<1>(a.weight, c, n);
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = r.get(i);
    } else if (a.w_dtype == QUADS_OUT_F32) {
        const Raw<0> r = load<0>(a.weight, c, n);
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = r.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = 1.0f;
    }
}

// h of eight channels, rounded to the residual's type.
template <int kX, int kR>
__device__ __forceinline__ void add_row(const void* x, const void* res, int64_t c, int64_t n,
                                        float* h) {
    const Raw<kX> a = load<kX>(x, c, n);
    if (kR == kNone) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) h[i] = a.get(i);
    } else {
        const Raw<kR & 1> b = load<kR & 1>(res, c, n);
        float s[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) s[i] = a.get(i) + b.get(i);
        const Raw<kR & 1> q = pack<kR & 1>(s);
#pragma unroll
        for (int i = 0; i < kPer; ++i) h[i] = q.get(i);
    }
}

template <int kX, int kR, int kOut>
__global__ __launch_bounds__(kThreads) void k_rms_rows(Args a) {
    __shared__ double s_part[kThreads / 64];
    __shared__ uint32_t s_max[kThreads / 64];
    uint32_t most = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void* x = row_at<kX>(a.x, t * a.ldx);
        const void* res = kR == kNone ? nullptr : row_at<kR & 1>(a.residual, t * a.ldr);
        void* sum = kR != kNone && a.sum ? row_at<kR & 1>(a.sum, t * a.H) : nullptr;
        double acc = 0.0;
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
            float h[kPer];
            add_row<kX, kR>(x, res, c, a.H - c, h);
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc = fma((double)h[i], (double)h[i], acc);
            if (kR != kNone && sum) store<kR & 1>(sum, c, a.H - c, pack<kR & 1>(h));
        }
        const double rstd = rsqrt(group_sum(acc, s_part) * a.inv_h + a.eps);
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
            const int64_t n = a.H - c;
            float h[kPer], w[kPer];
            if (kR != kNone && sum) {        // x or the residual may be gone: the sum took its place
                const Raw<kR & 1> q = load<kR & 1>(sum, c, n);
#pragma unroll
                for (int i = 0; i < kPer; ++i) h[i] = q.get(i);
            } else {
                add_row<kX, kR>(x, res, c, n, h);
            }
            load_weight(a, c, n, w);
            if (kOut == QUADS_OUT_MX_FP8) {
                uint32_t u[kPer], top = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    u[i] = upper((double)h[i] * rstd * (double)w[i]);
                    const uint32_t m = u[i] & 0x7FFFFFFFu;
                    top = m > top ? m : top;
                }
                // the block's other three threads (H % 32 == 0: all of them are here)
                uint32_t o = __shfl_xor(top, 1, 64);
                top = o > top ? o : top;
                o = __shfl_xor(top, 2, 64);
                top = o > top ? o : top;
                const int e = mx_exponent(top);
                float f[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) f[i] = mx_scaled(u[i], e);
                *reinterpret_cast<words2*>((uint8_t*)a.y + t * a.H + c) = mx_codes(f);
                if ((threadIdx.x & 3) == 0) a.scales[(t * a.H + c) / 32] = (uint8_t)(e + 127);
            } else {
                const float r = (float)rstd;
                float y[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) y[i] = h[i] * r * w[i];
                const Raw<kOut & 1> q = pack<kOut & 1>(y);
                store<kOut & 1>(row_at<kOut & 1>(a.y, t * a.H), c, n, q);
                if (kOut == QUADS_OUT_BF16 && a.amax_part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) most = pk_max_u16(most, q.q[0][i] & 0x7FFF7FFFu);
                }
            }
        }
    }
    if (kOut == QUADS_OUT_BF16 && a.amax_part) {
        uint32_t m = (most & 0xFFFFu) > (most >> 16) ? (most & 0xFFFFu) : (most >> 16);
#pragma unroll
        for (int off = 32; off; off >>= 1) {
            const uint32_t o = __shfl_xor(m, off, 64);
            m = o > m ? o : m;
        }
        if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kThreads / 64; ++i) m = s_max[i] > m ? s_max[i] : m;
            a.amax_part[blockIdx.x] = m;
        }
        if (blockIdx.x == 0)
            for (int64_t i = gridDim.x + threadIdx.x; i < a.amax_groups; i += kThreads)
                a.amax_part[i] = 0;
    }
}

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
__device__ __forceinline__ void load_weight(const GradArgs& a, int64_t c, int64_t n, float* w) {
    Args b;
    b.weight = a.weight;
    b.w_dtype = a.w_dtype;
    load_weight(b, c, n, w);
}

// (r, c) of each row.
template <int kG, int kH>
__global__ __launch_bounds__(kThreads) void k_rms_grad_stat(GradArgs a) {
    __shared__ double s_part[kThreads / 64];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void* g = row_at<kG>(a.g, t * a.H);
        const void* h = row_at<kH>(a.h, t * a.ldh);
        double sq = 0.0, dot = 0.0;
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
            const Raw<kG> gr = load<kG>(g, c, a.H - c);
            const Raw<kH> hr = load<kH>(h, c, a.H - c);
            float w[kPer];
            load_weight(a, c, a.H - c, w);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const double hd = hr.get(i);
                sq = fma(hd, hd, sq);
                dot = fma(hd, (double)(gr.get(i) * w[i]), dot);
            }
        }
        const double rd = rsqrt(group_sum(sq, s_part) * a.inv_h + a.eps);
        const double c = group_sum(dot, s_part) * a.inv_h * rd;
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
    load_weight(a, c, n, w);
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

constexpr int64_t kMaxGroups = 2048;         // work-groups of a forward call
inline int64_t row_groups(int64_t T) { return T < kMaxGroups ? T : kMaxGroups; }
// Runs of rows: one weight gradient's partial sum each.
inline int64_t grad_runs(int64_t T) { return T < 8 ? 1 : (T / 8 < 512 ? T / 8 : 512); }

template <int kX, int kR>
void launch(const Args& a, int out_dtype, hipStream_t s) {
    const dim3 grid((unsigned)row_groups(a.T)), block(kThreads);
    if (out_dtype == QUADS_OUT_F32)
        hipLaunchKernelGGL((k_rms_rows<kX, kR, QUADS_OUT_F32>), grid, block, 0, s, a);
    else if (out_dtype == QUADS_OUT_BF16)
        hipLaunchKernelGGL((k_rms_rows<kX, kR, QUADS_OUT_BF16>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_rms_rows<kX, kR, QUADS_OUT_MX_FP8>), grid, block, 0, s, a);
}

template <int kG, int kH>
void launch_grad(const GradArgs& a, hipStream_t s) {
    const dim3 block(kThreads);
    hipLaunchKernelGGL((k_rms_grad_stat<kG, kH>), dim3((unsigned)row_groups(a.T)), block, 0, s, a);
    const unsigned cols = (unsigned)((a.H + kThreads * kPer - 1) / (kThreads * kPer));
    hipLaunchKernelGGL((k_rms_grad_apply<kG, kH>), dim3(cols, (unsigned)a.runs), block, 0, s, a);
}

inline int check_sizes(int64_t T, int64_t H, int64_t ld) {
    if (T < 0 || T >= ((int64_t)1 << 31) || H < 1 || H >= kMaxH) return QUADS_ESHAPE;
    return ld < H || ld >= kMaxStride ? QUADS_ESHAPE : QUADS_OK;
}

}  // namespace norm
}  // namespace quads

using namespace quads;

extern "C" int64_t quads_rmsnorm_amax_groups(int64_t T, int64_t H) {
    if (norm::check_sizes(T, H, H) != QUADS_OK || T == 0) return 0;
    return norm::row_groups(T);
}

extern "C" int quads_rmsnorm(const void* x, int x_dtype, int64_t T, int64_t H, int64_t ldx,
                             const void* residual, int res_dtype, int64_t ldr, const void* weight,
                             int w_dtype, double eps, void* sum, void* y, int out_dtype,
                             uint8_t* scales, uint32_t* amax_part, int64_t amax_groups,
                             void* stream) {
    using namespace norm;
    if (int e = check_sizes(T, H, ldx)) return e;
    if (residual && (ldr < H || ldr >= kMaxStride)) return QUADS_ESHAPE;
    if (!ok_type(x_dtype) || (residual && !ok_type(res_dtype)) || (weight && !ok_type(w_dtype)))
        return QUADS_EINVAL;
    if (!ok_type(out_dtype) && out_dtype != QUADS_OUT_MX_FP8) return QUADS_EINVAL;
    if (out_dtype == QUADS_OUT_MX_FP8 && H % 32) return QUADS_ESHAPE;
    if (!(eps > 0.0) || !(eps <= 1.7976931348623157e308)) return QUADS_EINVAL;
    if (amax_part && (out_dtype != QUADS_OUT_BF16 || !ok_ptr4(amax_part))) return QUADS_EINVAL;
    if (sum && !residual) return QUADS_EINVAL;
    if (amax_part && amax_groups < quads_rmsnorm_amax_groups(T, H)) return QUADS_EWORKSPACE;
    if (T == 0) return QUADS_OK;
    if (!ok_ptr(x) || !ok_opt_ptr(residual) || !ok_opt_ptr(weight) || !ok_opt_ptr(sum) || !ok_ptr(y))
        return QUADS_EINVAL;
    if (out_dtype == QUADS_OUT_MX_FP8 && !ok_ptr(scales)) return QUADS_EINVAL;
    // in place only over rows that lie as the output's do
    if ((y == x && (ldx != H || out_dtype != x_dtype)) || y == sum ||
        (y == residual && (ldr != H || out_dtype != res_dtype)) ||
        (sum && ((sum == x && (ldx != H || res_dtype != x_dtype)) ||
                 (sum == residual && ldr != H))))
        return QUADS_EINVAL;
    Args a = {x,  residual, weight, sum, y,   scales, amax_part, T, H, ldx, residual ? ldr : 0,
              amax_groups, eps, 1.0 / (double)H, weight ? w_dtype : -1};
    hipStream_t s = (hipStream_t)stream;
    const int kind = (x_dtype == QUADS_OUT_BF16 ? 3 : 0) +
                     (!residual ? 2 : (res_dtype == QUADS_OUT_BF16 ? 1 : 0));
    switch (kind) {
        case 0: launch<0, 0>(a, out_dtype, s); break;
        case 1: launch<0, 1>(a, out_dtype, s); break;
        case 2: launch<0, kNone>(a, out_dtype, s); break;
        case 3: launch<1, 0>(a, out_dtype, s); break;
        case 4: launch<1, 1>(a, out_dtype, s); break;
        default: launch<1, kNone>(a, out_dtype, s); break;
    }
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

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
    if (!(eps > 0.0) || !(eps <= 1.7976931348623157e308)) return QUADS_EINVAL;
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
                  (T + runs - 1) / runs, (int)runs, eps, 1.0 / (double)H, weight ? w_dtype : -1,
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
