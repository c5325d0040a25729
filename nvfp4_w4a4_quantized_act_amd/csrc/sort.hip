// Tokens in packed (expert) order and back, and the gradient of the way back.
//
//   sort     out[pos[t, s]] = x[t]
//   unsort   out[t] = sum_s w[t, s] y[pos[t, s]]
//   gradient dy[pos[t, s]] = w[t, s] g[t],  dw[t, s] = <g[t], y[pos[t, s]]>
//
// Copies of rows: HBM bounds them.  Both directions go by token: the token's own
// row is then read (or written) once, and what is many rows, the packed side,
// once too, whole rows of it at places of its own.
#include "block.h"

namespace quads {
namespace sorting {

using namespace block;

constexpr int kThreads = 256;
constexpr int kMaxTopk = 64;

struct Args {
    const void* a;                           // x, y or g
    const void* y;                           // of the gradient
    void* out;                               // packed rows, token rows, or dy
    float* dw;
    const int32_t* pos;
    const float* w;
    int64_t T, H, ld, rows;
    int topk;
};

template <int kT>
__global__ __launch_bounds__(kThreads) void k_sort(Args a) {
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void* x = row_at<kT>(a.a, t * a.ld);
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
            const Raw<kT> r = load<kT>(x, c, a.H - c);
            for (int s = 0; s < a.topk; ++s) {
                const int64_t p = a.pos[t * a.topk + s];
                if (p >= 0 && p < a.rows) store<kT>(row_at<kT>(a.out, p * a.H), c, a.H - c, r);
            }
        }
    }
}

template <int kY, int kOut>
__global__ __launch_bounds__(kThreads) void k_unsort(Args a) {
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
            float acc[kPer] = {};
            for (int s = 0; s < a.topk; ++s) {
                const int64_t p = a.pos[t * a.topk + s];
                if (p < 0 || p >= a.rows) continue;
                const float w = a.w ? a.w[t * a.topk + s] : 1.0f;
                const Raw<kY> r = load<kY>(row_at<kY>(a.a, p * a.H), c, a.H - c);
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, r.get(i), acc[i]);
            }
            store<kOut>(row_at<kOut>(a.out, t * a.H), c, a.H - c, pack<kOut>(acc));
        }
    }
}

template <int kG, int kY>
__global__ __launch_bounds__(kThreads) void k_unsort_grad(Args a) {
    __shared__ float s_part[kMaxTopk][kThreads / 64];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void* g = row_at<kG>(a.a, t * a.H);
        for (int s = 0; s < a.topk; ++s) {
            const int64_t p = a.pos[t * a.topk + s];
            const bool have = p >= 0 && p < a.rows;
            float dot = 0.0f;
            if (have) {
                const float w = a.w ? a.w[t * a.topk + s] : 1.0f;
                for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kThreads * kPer) {
                    const int64_t n = a.H - c;
                    const Raw<kG> gr = load<kG>(g, c, n);
                    if (a.dw) {
                        const Raw<kY> yr = load<kY>(row_at<kY>(a.y, p * a.H), c, n);
#pragma unroll
                        for (int i = 0; i < kPer; ++i) dot = fmaf(gr.get(i), yr.get(i), dot);
                    }
                    if (a.out) {
                        float d[kPer];
#pragma unroll
                        for (int i = 0; i < kPer; ++i) d[i] = w * gr.get(i);
                        store<kY>(row_at<kY>(a.out, p * a.H), c, n, pack<kY>(d));
                    }
                }
            }
            if (a.dw) {
#pragma unroll
                for (int off = 32; off; off >>= 1) dot += __shfl_xor(dot, off, 64);
                if ((threadIdx.x & 63) == 0) s_part[s][threadIdx.x >> 6] = dot;
            }
        }
        if (a.dw) {
            __syncthreads();
            for (int s = threadIdx.x; s < a.topk; s += kThreads) {
                float v = 0.0f;
                for (int i = 0; i < kThreads / 64; ++i) v += s_part[s][i];
                a.dw[t * a.topk + s] = v;
            }
            __syncthreads();
        }
    }
}

constexpr int64_t kGroups = 1 << 20;         // work-groups of a call, at most
inline dim3 grid(int64_t T) { return dim3((unsigned)(T < kGroups ? T : kGroups)); }

inline int check(int64_t T, int64_t H, int64_t ld, int32_t topk, int64_t rows) {
    if (T < 0 || T >= ((int64_t)1 << 24) || H < 1 || H >= kMaxH || ld < H || ld >= kMaxStride)
        return QUADS_ESHAPE;
    if (topk < 1 || topk > kMaxTopk || rows < 0 || rows >= ((int64_t)1 << 31) ||
        T * topk >= ((int64_t)1 << 31))
        return QUADS_ESHAPE;
    return QUADS_OK;
}

}  // namespace sorting
}  // namespace quads

using namespace quads;

extern "C" int quads_moe_sort(const void* x, int dtype, int64_t T, int64_t H, int64_t ldx,
                              const int32_t* pos, int32_t topk, int64_t rows, void* out,
                              void* stream) {
    using namespace sorting;
    if (int e = check(T, H, ldx, topk, rows)) return e;
    if (!ok_type(dtype)) return QUADS_EINVAL;
    if (T == 0 || rows == 0) return QUADS_OK;
    if (!ok_ptr(x) || !ok_ptr4(pos) || !ok_ptr(out) || x == out) return QUADS_EINVAL;
    const Args a = {x, nullptr, out, nullptr, pos, nullptr, T, H, ldx, rows, topk};
    hipStream_t s = (hipStream_t)stream;
    if (dtype == QUADS_OUT_BF16)
        hipLaunchKernelGGL(k_sort<1>, grid(T), dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL(k_sort<0>, grid(T), dim3(kThreads), 0, s, a);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

extern "C" int quads_moe_unsort(const void* y, int y_dtype, int64_t rows, const int32_t* pos,
                                const float* topk_w, int64_t T, int32_t topk, int64_t H, void* out,
                                int out_dtype, void* stream) {
    using namespace sorting;
    if (int e = check(T, H, H, topk, rows)) return e;
    if (!ok_type(y_dtype) || !ok_type(out_dtype)) return QUADS_EINVAL;
    if (T == 0) return QUADS_OK;
    if ((rows > 0 && !ok_ptr(y)) || !ok_ptr4(pos) || !ok_opt4(topk_w) || !ok_ptr(out) || y == out)
        return QUADS_EINVAL;
    const Args a = {y, nullptr, out, nullptr, pos, topk_w, T, H, H, rows, topk};
    hipStream_t s = (hipStream_t)stream;
    const bool yb = y_dtype == QUADS_OUT_BF16, ob = out_dtype == QUADS_OUT_BF16;
    if (yb && ob) hipLaunchKernelGGL((k_unsort<1, 1>), grid(T), dim3(kThreads), 0, s, a);
    else if (yb) hipLaunchKernelGGL((k_unsort<1, 0>), grid(T), dim3(kThreads), 0, s, a);
    else if (ob) hipLaunchKernelGGL((k_unsort<0, 1>), grid(T), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_unsort<0, 0>), grid(T), dim3(kThreads), 0, s, a);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

extern "C" int quads_moe_unsort_backward(const void* g, int g_dtype, const void* y, int y_dtype,
                                         int64_t rows, const int32_t* pos, const float* topk_w,
                                         int64_t T, int32_t topk, int64_t H, void* dy, float* dw,
                                         void* stream) {
    using namespace sorting;
    if (int e = check(T, H, H, topk, rows)) return e;
    if (!ok_type(g_dtype) || !ok_type(y_dtype)) return QUADS_EINVAL;
    if (dw && !topk_w) return QUADS_EINVAL;
    if (T == 0 || (!dy && !dw)) return QUADS_OK;
    if (!ok_ptr(g) || (rows > 0 && dw && !ok_ptr(y)) || !ok_ptr4(pos) || !ok_opt4(topk_w) ||
        !ok_opt_ptr(dy) || !ok_opt4(dw) || dy == g)
        return QUADS_EINVAL;
    const Args a = {g, y, dy, dw, pos, topk_w, T, H, H, rows, topk};
    hipStream_t s = (hipStream_t)stream;
    const bool gb = g_dtype == QUADS_OUT_BF16, yb = y_dtype == QUADS_OUT_BF16;
    if (gb && yb) hipLaunchKernelGGL((k_unsort_grad<1, 1>), grid(T), dim3(kThreads), 0, s, a);
    else if (gb) hipLaunchKernelGGL((k_unsort_grad<1, 0>), grid(T), dim3(kThreads), 0, s, a);
    else if (yb) hipLaunchKernelGGL((k_unsort_grad<0, 1>), grid(T), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_unsort_grad<0, 0>), grid(T), dim3(kThreads), 0, s, a);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}
