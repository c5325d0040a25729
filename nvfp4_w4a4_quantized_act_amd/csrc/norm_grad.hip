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
    int64_t rows;                            // of a run of rows, or of a stretch
    int runs, wide;                          // work-groups of a stretch
    double eps, inv_h;
    int w_dtype, dx_dtype;
};

// ---- rows of up to 16384 channels: one read of g, h and g_sum, one write ----------------
//
// A row stays in the registers of the threads that share it (kLanes, or 64 n of them)
// between the two sums and dh, eight channels in each (kV = 2: sixteen; a few of its
// registers spill, and the weight read again for each row is slower: 2048 x 16384 bf16
// 69 us against 74.5).  A work-group holds several rows at once, up to 1024 threads, and
// takes more in turn: each thread keeps its channels' weight and their part of dweight in
// registers all the while, and a work-group leaves one partial dweight at its end.  The
// kernel runs at HBM's rate (16384 x 2048 bf16 with dweight 51 us, 5.3 TB/s; two kernels
// that each read g and h took four times as long); the next row's loads asked for before
// the sums bring nothing (57.8 against 57.6 us with the join).  bf16 rows of whole 16 bytes
// are read past the caches: 16384 x 2048 57.4 us / 55.1, 8192 x 4096 58.2 / 54.9, 65536 x
// 128 19.2 / 18.5; fp32's 32 bytes of a lane are two accesses to a line, 8192 x 8192 195 us
// against 217.
template <int kG, int kH, int kLanes, int kV, int kCut>
__global__ __launch_bounds__(1024) void k_rms_grad_held(GradArgs a, int lanes_) {
    __shared__ double s_sq[2][kMaxWaves], s_dot[2][kMaxWaves];
    __shared__ __align__(16) float s_acc[kV == 1 ? 1024 * kPer : 1];
    const int lanes = kLanes ? kLanes : lanes_;
    const int rows = (int)blockDim.x / lanes;
    const int row = threadIdx.x / lanes, lane = threadIdx.x - row * lanes;
    Piece p[kV];
    float w[kV][kPer], acc[kV][kPer];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        p[j] = piece<kCut>((j * lanes + lane) * kPer, (int)a.H);
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[j][i] = acc[j][i] = 0.0f;
        if (p[j].n > 0) load_weight(a.weight, a.w_dtype, p[j].at, p[j].n, w[j]);
    }
    int set = 0;
    const int64_t stretch = blockIdx.x / (unsigned)a.wide, first = stretch * a.rows;
    const int64_t end = first + a.rows < a.T ? first + a.rows : a.T;
    for (int64_t t0 = first + (blockIdx.x - stretch * a.wide) * rows; t0 < end;
         t0 += (int64_t)a.wide * rows) {
        const int64_t t = t0 + row;
        const bool live = t < a.T;
        Raw<kG> g[kV];
        Raw<kH> h[kV], s[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            g[j] = Raw<kG>{};
            h[j] = s[j] = Raw<kH>{};
            if (live && p[j].n > 0) {
                g[j] = load<kG, kCut != kTiny, kG && kCut == kEven>(row_at<kG>(a.g, t * a.H),
                                                                    p[j].at, p[j].n);
                h[j] = load<kH, kCut != kTiny, kH && kCut == kEven>(row_at<kH>(a.h, t * a.ldh),
                                                                    p[j].at, p[j].n);
                if (a.g_sum)
                    s[j] = load<kH, kCut != kTiny, kH && kCut == kEven>(
                        row_at<kH>(a.g_sum, t * a.H), p[j].at, p[j].n);
            }
        }
        double sq = 0.0, dot = 0.0;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (kCut == kOdd && i < p[j].from) continue;
                const double hd = h[j].get(i);
                sq = fma(hd, hd, sq);
                dot = fma(hd, (double)(g[j].get(i) * w[j][i]), dot);
            }
        }
        if constexpr (kLanes == 0) {         // as group_sum, over the row's waves
            sq = lanes_sum<64>(sq);
            dot = lanes_sum<64>(dot);
            const int wave = threadIdx.x >> 6, n = lanes >> 6;
            if ((threadIdx.x & 63) == 0) {
                s_sq[set][wave] = sq;
                s_dot[set][wave] = dot;
            }
            __syncthreads();
            const int i = threadIdx.x & (kMaxWaves - 1);
            sq = lanes_sum<kMaxWaves>(i < n ? s_sq[set][row * n + i] : 0.0);
            dot = lanes_sum<kMaxWaves>(i < n ? s_dot[set][row * n + i] : 0.0);
            set ^= 1;
        } else {
            sq = lanes_sum<kLanes>(sq);
            dot = lanes_sum<kLanes>(dot);
        }
        const double rd = rsqrt(sq * a.inv_h + a.eps);
        const float r = (float)rd, cn = (float)(dot * a.inv_h * rd);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            if (!live || p[j].n <= 0) continue;
            float d[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float n = h[j].get(i) * r;
                if (kCut != kOdd || i >= p[j].from) acc[j][i] = fmaf(g[j].get(i), n, acc[j][i]);
                d[i] = r * fmaf(-cn, n, g[j].get(i) * w[j][i]);
            }
            if (a.g_sum) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) d[i] += s[j].get(i);
            }
            if (a.dres)
                store<kH, kCut != kTiny>(row_at<kH>(a.dres, t * a.H), p[j].at, p[j].n, pack<kH>(d));
            if (a.dx_dtype == QUADS_OUT_BF16)
                store<1, kCut != kTiny>(row_at<1>(a.dx, t * a.H), p[j].at, p[j].n, pack<1>(d));
            else
                store<0, kCut != kTiny>(row_at<0>(a.dx, t * a.H), p[j].at, p[j].n, pack<0>(d));
        }
    }
    if (!a.part) return;
    if (kV == 1 && rows > 1) {               // the rows' parts, in order
        Raw<0> mine = pack<0>(acc[0]);
        words4* at = reinterpret_cast<words4*>(s_acc + threadIdx.x * kPer);
        at[0] = mine.q[0];
        at[1] = mine.q[1];
        __syncthreads();
        if (row > 0) return;
        for (int o = 1; o < rows; ++o) {
            const float* other = s_acc + (o * lanes + lane) * kPer;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[0][i] += other[i];
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        if (p[j].n <= 0) continue;
        if (p[j].from == 0) {
            store<0>(part, p[j].at, p[j].n, pack<0>(acc[j]));
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i >= p[j].from) part[p[j].at + i] = acc[j][i];
        }
    }
}

// ---- rows of any length: two reads --------------------------------------------------------
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
// rows of a run; `cols` neighbouring work-groups have one run.  Each value of g and
// g_sum is read before its place is written, by the same thread.
template <int kG, int kH>
__global__ __launch_bounds__(kThreads) void k_rms_grad_apply(GradArgs a, unsigned cols) {
    const unsigned run = blockIdx.x / cols;
    const int64_t c = ((int64_t)(blockIdx.x - run * cols) * kThreads + threadIdx.x) * kPer;
    if (c >= a.H) return;
    const int64_t n = a.H - c, t0 = run * a.rows;
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
    if (a.part) store<0>(a.part + run * a.H, c, n, pack<0>(acc));
}

// dweight from the partial sums of `runs` work-groups or runs of rows: 16 channels a
// work-group, the runs over its 64 groups of 16 threads, joined in fp64 (64 channels a work-group
// of 16 waves: 4096 x 2048 bf16 21.4 us with the gradient, 20.9 so).
__global__ __launch_bounds__(1024) void k_rms_join_weight(const float* part, int runs, int64_t H,
                                                          void* dweight, int bf16) {
    __shared__ double s_sum[kMaxWaves][16];
    const int i = threadIdx.x & 15;
    const int64_t c = (int64_t)blockIdx.x * 16 + i;
    double s = 0.0;
    if (c < H) {
#pragma unroll 4
        for (int k = threadIdx.x >> 4; k < runs; k += 64) s += (double)part[k * H + c];
    }
    s = both_sum<32>(both_sum<16>(s));
    if ((threadIdx.x & 63) < 16) s_sum[threadIdx.x >> 6][i] = s;
    __syncthreads();
    if (threadIdx.x >= 16 || c >= H) return;
#pragma unroll
    for (int k = 1; k < kMaxWaves; ++k) s += s_sum[k][i];
    if (bf16) ((uint16_t*)dweight)[c] = (uint16_t)bf16_bits((float)s, 0.0f);
    else ((float*)dweight)[c] = (float)s;
}

// ------------------------------------------------------------------- host --
struct GradShape {
    int lanes, v, threads;                   // v 0: two reads
};
// A work-group of up to 1024 threads holds as many rows at once as leave a row for each of
// 256 work-groups.
inline GradShape grad_shape(int64_t T, int64_t H) {
    int lanes = 8;
    while (lanes < 64 && lanes * kPer < H) lanes *= 2;
    if (lanes * kPer < H) lanes = (int)((H + 511) / 512 * 64);
    if (H <= 8192) {
        const int64_t most = 1024 / lanes, rows = (T + 255) / 256;
        int r = (int)(rows < most ? rows : most);
        while (r * lanes % 64) ++r;
        return {lanes, 1, r * lanes};
    }
    if (H <= 16384) return {(int)((H + 1023) / 1024 * 64), 2, (int)((H + 1023) / 1024 * 64)};
    return {0, 0, 0};
}
// Work-groups (held rows) or runs of rows: a partial dweight each.  One work-group of 1024
// threads a CU, two of up to 768 where each still has 16 rows (8192 x 5000 bf16 73 us
// against 80, 777 x 5001 fp32 26.7 / 23.8: more partial sums); two of 1024 would not fit
// with their 80 registers, and took 16384 x 2048 bf16 from 57.6 to 59.1 us.  All with the
// same number of rows, nearly.  Where a thread would add up more than kChain rows in fp32,
// whose rounding would grow with T (512 rows off by up to 124 * 2^-24, 64 by 64), the rows
// are cut into stretches, one after another, each with work-groups of its own (every
// work-group's rows over all of T instead: 262144 x 4096 bf16 1735 us against 1579).
constexpr int64_t kMaxGroups = 2048, kChain = 64;
struct Runs {
    int64_t stretches, wide, turns;          // work-groups of a stretch, and the rows in turn of each
};
inline Runs grad_stretches(int64_t T, int64_t H) {
    const GradShape p = grad_shape(T, H);
    if (!p.v) {
        const int64_t n = T < 8 ? 1 : (T / 8 < 512 ? T / 8 : 512), least = (T + kChain - 1) / kChain;
        return {1, n > least ? n : least, 0};
    }
    const int64_t rows = p.threads / p.lanes, n = (T + rows - 1) / rows;
    const int64_t most = p.threads <= 768 && n >= 8192 ? 512 : 256;
    const int64_t stretches = (n + most * kChain - 1) / (most * kChain);
    const int64_t each = (n + stretches - 1) / stretches, turns = (each + most - 1) / most;
    return {stretches, (each + turns - 1) / turns, turns};
}
inline int64_t grad_runs(int64_t T, int64_t H) {
    const Runs r = grad_stretches(T, H);
    return r.stretches * r.wide;
}

template <int kG, int kH>
void launch_grad(const GradArgs& a, hipStream_t s) {
    const GradShape p = grad_shape(a.T, a.H);
    const Cut cut = cut_of(a.H);
#define QUADS_HELD(L, V, C)                                                               \
    if (p.v == V && (p.lanes < 128 ? p.lanes : 0) == L && cut == C) {                     \
        hipLaunchKernelGGL((k_rms_grad_held<kG, kH, L, V, C>), dim3((unsigned)a.runs),    \
                           dim3(p.threads), 0, s, a, p.lanes);                            \
        return;                                                                           \
    }
#define QUADS_HELD_ANY(L, V) QUADS_HELD(L, V, kEven) QUADS_HELD(L, V, kOdd)
    QUADS_HELD(8, 1, kTiny)
    QUADS_HELD_ANY(8, 1)
    QUADS_HELD_ANY(16, 1)
    QUADS_HELD_ANY(32, 1)
    QUADS_HELD_ANY(64, 1)
    QUADS_HELD_ANY(0, 1)
    QUADS_HELD_ANY(0, 2)
#undef QUADS_HELD_ANY
#undef QUADS_HELD
    const dim3 block(kThreads);
    const int64_t rows = a.T < kMaxGroups ? a.T : kMaxGroups;
    hipLaunchKernelGGL((k_rms_grad_stat<kG, kH>), dim3((unsigned)rows), block, 0, s, a);
    const unsigned cols = (unsigned)((a.H + kThreads * kPer - 1) / (kThreads * kPer));
    const dim3 grid(cols * (unsigned)a.runs);
    hipLaunchKernelGGL((k_rms_grad_apply<kG, kH>), grid, block, 0, s, a, cols);
}

}  // namespace norm
}  // namespace quads

using namespace quads;

extern "C" size_t quads_rmsnorm_backward_ws(int64_t T, int64_t H, int want_dweight) {
    if (norm::check_sizes(T, H, H) != QUADS_OK || T == 0) return 0;
    return (norm::grad_shape(T, H).v ? 0 : align_up((size_t)T * 8, 256)) +
           (want_dweight ? align_up((size_t)norm::grad_runs(T, H) * H * 4, 256) : 0);
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
    const dim3 join((unsigned)((H + 15) / 16));
    if (T == 0) {                            // no rows: their sum is 0
        if (dweight) {
            hipLaunchKernelGGL(k_rms_join_weight, join, dim3(1024), 0, s, nullptr, 0, H, dweight,
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
    const GradShape p = grad_shape(T, H);
    const Runs r = grad_stretches(T, H);
    const int64_t runs = r.stretches * r.wide;
    const int64_t rows = p.v ? r.turns * r.wide * (p.threads / p.lanes) : (T + runs - 1) / runs;
    const size_t stat = p.v ? 0 : align_up((size_t)T * 8, 256);
    float* part = dweight ? (float*)((char*)ws + stat) : nullptr;
    GradArgs a = {g, h, weight, g_sum, dx, dres, (float2*)ws, part, T, H, ldh,
                  rows, (int)runs, (int)r.wide, eps, 1.0 / (double)H,
                  weight ? w_dtype : kNoWeight, dx_dtype};
    const bool gb = g_dtype == QUADS_OUT_BF16, hb = h_dtype == QUADS_OUT_BF16;
    if (gb && hb) launch_grad<1, 1>(a, s);
    else if (gb) launch_grad<1, 0>(a, s);
    else if (hb) launch_grad<0, 1>(a, s);
    else launch_grad<0, 0>(a, s);
    QUADS_CHECK_LAUNCH();
    if (dweight) {
        hipLaunchKernelGGL(k_rms_join_weight, join, dim3(1024), 0, s, a.part, (int)runs, H,
                           dweight, w_bf16);
        QUADS_CHECK_LAUNCH();
    }
    return QUADS_OK;
}
