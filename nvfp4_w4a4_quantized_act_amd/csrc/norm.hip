// Residual addition with the root-mean-square norm (formulas in norm.h).
//
// Bytes bound it: x and the residual are read once, the sum and y written once.  A row
// stays in the registers of the lanes that share it between the sum of its squares and
// the product (k_rms_held); only rows beyond 32768 channels are read again (k_rms_long).
#include "norm.h"

namespace quads {
namespace norm {

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
    int w_dtype, out_dtype;
};

// h of eight channels, rounded to the residual's type.
template <int kX, int kR>
__device__ __forceinline__ void add(const Raw<kX>& a, const Raw<kR & 1>& b, float* h) {
    if (kR == kNone) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) h[i] = a.get(i);
    } else {
        float s[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) s[i] = a.get(i) + b.get(i);
        const Raw<kR & 1> q = pack<kR & 1>(s);
#pragma unroll
        for (int i = 0; i < kPer; ++i) h[i] = q.get(i);
    }
}

// y of eight channels from h, stored; `most`: the largest magnitude's bits so far (bf16
// pairs), for amax_part.  MX FP8: the four threads of a block of 32 channels are all here
// or none of them (H % 32 == 0).
template <int kFp8, bool kWhole = false>
__device__ __forceinline__ void finish(const Args& a, int64_t t, int64_t c, int n, const float* h,
                                       const float* w, double rstd, uint32_t& most) {
    if (kFp8) {
        uint32_t u[kPer], top = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            u[i] = upper((double)h[i] * rstd * (double)w[i]);
            top = larger(top, u[i] & 0x7FFFFFFFu);
        }
        const int e = mx_exponent(lanes_max<4>(top));
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
        if (a.out_dtype == QUADS_OUT_BF16) {
            const Raw<1> q = pack<1>(y);
            store<1, kWhole>(row_at<1>(a.y, t * a.H), c, n, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) most = pk_max_u16(most, q.q[0][i] & 0x7FFF7FFFu);
        } else {
            store<0, kWhole>(row_at<0>(a.y, t * a.H), c, n, pack<0>(y));
        }
    }
}

// The work-group's largest magnitude, and zeros behind the work-groups.
__device__ __forceinline__ void leave_amax(const Args& a, uint32_t most) {
    __shared__ uint32_t s_max[kMaxWaves];
    const uint32_t m = lanes_max<64>(larger(most & 0xFFFFu, most >> 16));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t all = s_max[0];
        for (int i = 1; i < (int)(blockDim.x >> 6); ++i) all = larger(all, s_max[i]);
        a.amax_part[blockIdx.x] = all;
    }
    if (blockIdx.x == 0)
        for (int64_t i = gridDim.x + threadIdx.x; i < a.amax_groups; i += blockDim.x)
            a.amax_part[i] = 0;
}

// kLanes threads to a row (0: the whole work-group), kV times eight channels in each.
template <int kX, int kR, int kFp8, int kLanes, int kV, int kCut>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_rms_held(Args a) {
    __shared__ double s_part[2][kMaxWaves];
    const int lanes = kLanes ? kLanes : (int)blockDim.x, rows = kLanes ? 256 / kLanes : 1;
    const int lane = kLanes ? threadIdx.x % kLanes : threadIdx.x;
    Piece p[kV];
    float w[kV][kPer];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        p[j] = piece<kCut>((j * lanes + lane) * kPer, (int)a.H);
        if (p[j].n > 0) load_weight(a.weight, a.w_dtype, p[j].at, p[j].n, w[j]);
    }
    uint32_t most = 0;
    int set = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += (int64_t)gridDim.x * rows) {
        const int64_t t = t0 + (kLanes ? threadIdx.x / kLanes : 0);
        const bool live = kLanes == 0 || t < a.T;
        const void* x = row_at<kX>(a.x, t * a.ldx);
        const void* res = kR == kNone ? nullptr : row_at<kR & 1>(a.residual, t * a.ldr);
        Raw<kX> xr[kV];
        Raw<kR & 1> rr[kV];
        float h[kV][kPer];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            xr[j] = Raw<kX>{};
            if (kR != kNone) rr[j] = Raw<kR & 1>{};
            if (live && p[j].n > 0) {
                xr[j] = load<kX, kCut != kTiny>(x, p[j].at, p[j].n);
                if (kR != kNone) rr[j] = load<kR & 1, kCut != kTiny>(res, p[j].at, p[j].n);
            }
        }
        double acc = 0.0;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            add<kX, kR>(xr[j], rr[j], h[j]);
            if (kCut != kOdd || p[j].from == 0) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc = fma((double)h[j][i], (double)h[j][i], acc);
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (i >= p[j].from) acc = fma((double)h[j][i], (double)h[j][i], acc);
            }
        }
        // The sum may stand in the residual's place and y in x's: of a channel that two
        // threads share (kOdd), both have read it when one writes, behind the rows' sum.
        // Otherwise the stores go out before it (8192 x 5000 bf16: 64.5 us against 68).
        auto store_sum = [&] {
#pragma unroll
            for (int j = 0; j < kV; ++j)
                if (live && p[j].n > 0)
                    store<kR & 1, kCut != kTiny>(row_at<kR & 1>(a.sum, t * a.H), p[j].at, p[j].n,
                                                 pack<kR & 1>(h[j]));
        };
        if (kR != kNone && kCut != kOdd && a.sum) store_sum();
        double total;
        if constexpr (kLanes == 0) total = group_sum(acc, s_part, set);
        else total = lanes_sum<kLanes>(acc);
        set ^= 1;
        if (kR != kNone && kCut == kOdd && a.sum) store_sum();
        const double rstd = rsqrt(total * a.inv_h + a.eps);
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (live && p[j].n > 0)
                finish<kFp8, kCut != kTiny>(a, t, p[j].at, p[j].n, h[j], w[j], rstd, most);
    }
    if (!kFp8 && a.amax_part) leave_amax(a, most);
}

// Rows of any length, read twice.
constexpr int kLongThreads = 1024;
template <int kX, int kR, int kFp8>
__global__ __launch_bounds__(kLongThreads) void k_rms_long(Args a) {
    __shared__ double s_part[2][kMaxWaves];
    uint32_t most = 0;
    int set = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const void* x = row_at<kX>(a.x, t * a.ldx);
        const void* res = kR == kNone ? nullptr : row_at<kR & 1>(a.residual, t * a.ldr);
        void* sum = kR != kNone && a.sum ? row_at<kR & 1>(a.sum, t * a.H) : nullptr;
        double acc = 0.0;
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kLongThreads * kPer) {
            float h[kPer];
            const Raw<kX> xr = load<kX>(x, c, a.H - c);
            Raw<kR & 1> rr;
            if (kR != kNone) rr = load<kR & 1>(res, c, a.H - c);
            add<kX, kR>(xr, rr, h);
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc = fma((double)h[i], (double)h[i], acc);
            if (kR != kNone && sum) store<kR & 1>(sum, c, a.H - c, pack<kR & 1>(h));
        }
        const double total = group_sum(acc, s_part, set);
        set ^= 1;
        const double rstd = rsqrt(total * a.inv_h + a.eps);
        for (int64_t c = (int64_t)threadIdx.x * kPer; c < a.H; c += kLongThreads * kPer) {
            const int64_t n = a.H - c;
            float h[kPer], w[kPer];
            if (kR != kNone && sum) {        // it may have taken x's or the residual's place
                const Raw<kR & 1> q = load<kR & 1>(sum, c, n);
#pragma unroll
                for (int i = 0; i < kPer; ++i) h[i] = q.get(i);
            } else {
                const Raw<kX> xr = load<kX>(x, c, n);
                Raw<kR & 1> rr;
                if (kR != kNone) rr = load<kR & 1>(res, c, n);
                add<kX, kR>(xr, rr, h);
            }
            load_weight(a.weight, a.w_dtype, c, n, w);
            finish<kFp8>(a, t, c, (int)(n < kPer ? n : kPer), h, w, rstd, most);
        }
    }
    if (!kFp8 && a.amax_part) leave_amax(a, most);
}

// ------------------------------------------------------------------- host --
// Lanes and channels per lane by the row's length: up to 1024 channels part of a wave or
// a wave, above that a work-group of as many waves as the row fills with eight channels a
// thread, above 8192 with more in each.  Rows of 2048 and 4096 in a wave of their own (32
// and 64 channels a lane) take 16384 x 2048 bf16 51.7 us against 49.3, 16384 x 4096 into
// FP8 138 against 106, and 64 x 4096 7.0 against 3.5; a work-group for rows below 1024
// 16384 x 1000 bf16 16.4 against 14.1.
struct Shape {
    int lanes, v, threads;                   // 0 lanes: the work-group; v 0: k_rms_long
};
inline Shape shape_of(int64_t H) {
    if (H <= 64) return {8, 1, 256};
    if (H <= 128) return {16, 1, 256};
    if (H <= 256) return {32, 1, 256};
    if (H <= 512) return {64, 1, 256};
    if (H <= 1024) return {64, 2, 256};
    for (int v = 1; v <= 4; v *= 2)
        if (H <= 8192 * v) return {0, v, (int)((H + 512 * v - 1) / (512 * v) * 64)};
    return {0, 0, kLongThreads};
}
// Work-groups of a call: up to 2048, each with several rows in turn, which then read the
// weight once; calls that move more than the caches hold are faster with the rows in
// order, a work-group for each (16384 x 4096 bf16: 92.5 us against 103.5, 16384 x 2048
// 48.6 / 52.8, 4096 x 2048 15.6 / 14.7, 131072 x 128 15.5 / 13.7; at most 2^21 of them,
// a launch has fewer than 2^32 threads).  Partial maxima are read by every work-group of
// the quantizer: with them never more than 2048.
constexpr int64_t kMaxGroups = 2048, kManyBytes = (int64_t)192 << 20;
inline int64_t groups_of(int64_t T, int64_t H, int64_t bytes) {
    const Shape s = shape_of(H);
    const int64_t rows = s.lanes ? s.threads / s.lanes : 1;
    const int64_t n = (T + rows - 1) / rows;
    return n < kMaxGroups || (bytes > kManyBytes && n < ((int64_t)1 << 21)) ? n : kMaxGroups;
}

template <int kX, int kR, int kFp8>
void launch(const Args& a, hipStream_t s) {
    const int64_t bytes =
        a.T * a.H * ((kX ? 2 : 4) + (kR == kNone ? 0 : (kR ? 2 : 4) * (a.sum ? 2 : 1)) +
                     (kFp8 ? 1 : a.out_dtype == QUADS_OUT_BF16 ? 2 : 4));
    const dim3 grid((unsigned)groups_of(a.T, a.H, a.amax_part ? 0 : bytes));
    const Shape p = shape_of(a.H);
    const Cut cut = cut_of(a.H);
#define QUADS_HELD(L, V, C)                                                             \
    if (p.lanes == L && p.v == V && cut == C) {                                         \
        hipLaunchKernelGGL((k_rms_held<kX, kR, kFp8, L, V, C>), grid, dim3(p.threads), 0, s, a); \
        return;                                                                         \
    }
#define QUADS_HELD_ANY(L, V)  \
    QUADS_HELD(L, V, kEven)   \
    if constexpr (!kFp8) {    \
        QUADS_HELD(L, V, kOdd) \
    }
    if constexpr (!kFp8) {
        QUADS_HELD(8, 1, kTiny)
    }
    QUADS_HELD_ANY(8, 1)
    QUADS_HELD_ANY(16, 1)
    QUADS_HELD_ANY(32, 1)
    QUADS_HELD_ANY(64, 1)
    QUADS_HELD_ANY(64, 2)
    QUADS_HELD_ANY(0, 1)
    QUADS_HELD_ANY(0, 2)
    QUADS_HELD_ANY(0, 4)
#undef QUADS_HELD_ANY
#undef QUADS_HELD
    hipLaunchKernelGGL((k_rms_long<kX, kR, kFp8>), grid, dim3(kLongThreads), 0, s, a);
}
template <int kX, int kR>
void launch(const Args& a, hipStream_t s) {
    if (a.out_dtype == QUADS_OUT_MX_FP8) launch<kX, kR, 1>(a, s);
    else launch<kX, kR, 0>(a, s);
}

}  // namespace norm
}  // namespace quads

using namespace quads;

extern "C" int64_t quads_rmsnorm_amax_groups(int64_t T, int64_t H) {
    if (norm::check_sizes(T, H, H) != QUADS_OK || T == 0) return 0;
    return norm::groups_of(T, H, 0);
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
    if (!ok_eps(eps)) return QUADS_EINVAL;
    if (amax_part && (out_dtype != QUADS_OUT_BF16 || !ok_ptr4(amax_part))) return QUADS_EINVAL;
    if (sum && !residual) return QUADS_EINVAL;
    if (amax_part && amax_groups < quads_rmsnorm_amax_groups(T, H)) return QUADS_EWORKSPACE;
    if (T == 0) return QUADS_OK;
    if (!ok_ptr(x) || !ok_opt_ptr(residual) || !ok_opt_ptr(weight) || !ok_opt_ptr(sum) ||
        !ok_ptr(y))
        return QUADS_EINVAL;
    if (out_dtype == QUADS_OUT_MX_FP8 && !ok_ptr(scales)) return QUADS_EINVAL;
    // in place only over rows that lie as the output's do
    if ((y == x && (ldx != H || out_dtype != x_dtype)) || y == sum ||
        (y == residual && (ldr != H || out_dtype != res_dtype)) ||
        (sum && ((sum == x && (ldx != H || res_dtype != x_dtype)) ||
                 (sum == residual && ldr != H))))
        return QUADS_EINVAL;
    Args a = {x,  residual, weight, sum, y,   scales, amax_part, T, H, ldx, residual ? ldr : 0,
              amax_groups, eps, 1.0 / (double)H, weight ? w_dtype : kNoWeight, out_dtype};
    hipStream_t s = (hipStream_t)stream;
    const int kind = (x_dtype == QUADS_OUT_BF16 ? 3 : 0) +
                     (!residual ? 2 : (res_dtype == QUADS_OUT_BF16 ? 1 : 0));
    switch (kind) {
        case 0: launch<0, 0>(a, s); break;
        case 1: launch<0, 1>(a, s); break;
        case 2: launch<0, kNone>(a, s); break;
        case 3: launch<1, 0>(a, s); break;
        case 4: launch<1, 1>(a, s); break;
        default: launch<1, kNone>(a, s); break;
    }
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}
