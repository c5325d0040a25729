// W4A16 grouped product for few rows per expert (include/quads_head.h): bf16
// activations times NVFP4 weights, arXiv 2607.15810, Eq. (12).
#include "common.h"
#include "gemm_tiles.h"
#include "../../include/quads_head.h"

namespace quads {
namespace w4a16 {

struct Args {
    const uint16_t* x; const int32_t* row_token; int64_t rows; int64_t K;
    const uint8_t* w_nib; const uint8_t* w_scale; const float* w_ts; const int32_t* offsets;
    int E; int64_t N;
    int out_bf16; void* out;
};

// Dot product of the activation row with weight row n of expert e, by a wave.
__device__ __forceinline__ float dot(const Args& a, const uint16_t* x, int e, int64_t n) {
    const int lane = threadIdx.x & 63;
    const uint8_t* w = a.w_nib + ((int64_t)e * a.N + n) * (a.K / 2);
    const uint8_t* sc = a.w_scale + ((int64_t)e * a.N + n) * (a.K / kBlock);
    float acc = 0.0f;
    for (int64_t b = lane; b < a.K / kBlock; b += 64) {
        float s = 0.0f;
        for (int h = 0; h < 2; ++h) {
            float v[8];
            decode8(reinterpret_cast<const uint32_t*>(w)[2 * b + h], v);
            for (int i = 0; i < 8; ++i)
                s = __builtin_fmaf(v[i], bf16_to_f32(x[kBlock * b + 8 * h + i]), s);
        }
        acc = __builtin_fmaf(s, e4m3_value(sc[b]), acc);
    }
    for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o);
    return acc * a.w_ts[e];
}

// One wave per output feature, over the packed rows in turn.
template <int kEpi>
__global__ __launch_bounds__(256) void k_gemv(Args a) {
    const int64_t ncols = kEpi == QUADS_EPI_SWIGLU ? a.N / 2 : a.N;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= ncols) return;
    int e = 0;
    for (int64_t p = 0; p < a.rows; ++p) {
        if (a.offsets)
            while (p >= a.offsets[e + 1]) ++e;
        const int64_t row = a.row_token ? a.row_token[p] : p;
        const uint16_t* x = a.x + row * a.K;
        float y = dot(a, x, e, n);
        if (kEpi == QUADS_EPI_SWIGLU) y = silu_mul(y, dot(a, x, e, n + ncols));
        if ((threadIdx.x & 63) == 0) {
            if (a.out_bf16)
                ((uint16_t*)a.out)[p * ncols + n] = __builtin_bit_cast(uint16_t, (__bf16)y);
            else
                ((float*)a.out)[p * ncols + n] = y;
        }
    }
}

}  // namespace w4a16
}  // namespace quads

using namespace quads;

extern "C" size_t quads_moe_w4a16_gemv_ws(int64_t rows, int64_t K, int32_t E, int64_t N) {
    (void)rows; (void)K; (void)E; (void)N;
    return 0;
}

extern "C" int quads_moe_w4a16_gemv(const uint16_t* x, const int32_t* row_token, int64_t rows,
                                    int64_t K, const uint8_t* w_nib, const uint8_t* w_scale,
                                    const float* w_ts, const int32_t* offsets, int32_t E,
                                    int64_t N, int epilogue, int out_dtype, void* out, void* ws,
                                    size_t ws_bytes, void* stream) {
    if (rows < 0 || rows >= ((int64_t)1 << 31) || K <= 0 || K % kBlock || K >= ((int64_t)1 << 30) ||
        E < 1 || E > 4096 || N < 1 || N >= ((int64_t)1 << 30))
        return QUADS_ESHAPE;
    if (epilogue != QUADS_EPI_NONE && epilogue != QUADS_EPI_SWIGLU) return QUADS_EINVAL;
    if (out_dtype != QUADS_OUT_F32 && out_dtype != QUADS_OUT_BF16) return QUADS_EINVAL;
    if (epilogue == QUADS_EPI_SWIGLU && out_dtype != QUADS_OUT_BF16) return QUADS_EINVAL;
    if (epilogue == QUADS_EPI_SWIGLU && N % 2) return QUADS_ESHAPE;
    if (offsets == nullptr && E != 1) return QUADS_EINVAL;
    if (rows == 0) return QUADS_OK;
    if (!ok_opt_ptr(offsets) || !ok_opt_ptr(row_token)) return QUADS_EINVAL;
    if (!ok_ptr(x) || !ok_ptr(w_nib) || !ok_ptr(w_scale) || !ok_ptr(w_ts) || !ok_ptr(out))
        return QUADS_EINVAL;
    const size_t need = quads_moe_w4a16_gemv_ws(rows, K, E, N);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return QUADS_EWORKSPACE;
    const w4a16::Args a{x, row_token, rows, K, w_nib, w_scale, w_ts, offsets, (int)E, N,
                        out_dtype == QUADS_OUT_BF16, out};
    const int64_t ncols = epilogue == QUADS_EPI_SWIGLU ? N / 2 : N;
    const dim3 grid((unsigned)((ncols + 3) / 4)), block(256);
    if (epilogue == QUADS_EPI_SWIGLU)
        hipLaunchKernelGGL(w4a16::k_gemv<QUADS_EPI_SWIGLU>, grid, block, 0, (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL(w4a16::k_gemv<QUADS_EPI_NONE>, grid, block, 0, (hipStream_t)stream, a);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}
