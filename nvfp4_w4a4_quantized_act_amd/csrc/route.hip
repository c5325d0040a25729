// Routing: the topk experts with the largest logits of each token, their weights,
// and the weights' gradient.
//
//   p = softmax(z),  w_i = p_{id_i}, or that divided by the sum over the topk
//   renorm 0: dz_v = a_i [v = id_i] - p_v A,   a_i = g_i w_i, A = sum a_i
//   renorm 1: dz_v = a_i - w_i A at v = id_i
//
// A wave per token, its logits in registers (logit e in lane e % 64).  The order
// is by one signed number per logit: the bits of a float, the lower 31 turned
// over where it is negative.  The wave takes the largest number topk times.
#include "block.h"

namespace quads {
namespace routing {

using namespace block;

constexpr int kThreads = 256;
constexpr int kMaxE = 4096, kMaxTopk = 64;
constexpr int kGone = INT32_MIN;             // below every logit's number

struct Args {
    const void* z;
    int32_t* ids;
    float* w;
    const float* g;
    void* dz;
    int64_t T, ld;
    int E, topk, renorm;
};

__device__ __forceinline__ float logit(const void* z, int bf16, int64_t at) {
    return bf16 ? bf16_to_f32(((const uint16_t*)z)[at]) : ((const float*)z)[at];
}
// z + 0 makes -0 a 0; a NaN of either sign stands above everything.
__device__ __forceinline__ int order_of(float z) {
    const int b = (int)__float_as_uint(z + 0.0f);
    return z != z ? INT32_MAX : b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int k) {
    return __uint_as_float((uint32_t)(k ^ ((k >> 31) & 0x7FFFFFFF)));
}
__device__ __forceinline__ int wave_max(int v) {
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const int o = __shfl_xor(v, off, 64);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
// exp(z - m), 0 for a masked logit even where nothing else is left.
__device__ __forceinline__ float term(float z, float m) {
    return z == -INFINITY ? 0.0f : expf(z - m);
}

template <int kBf16, int kV>
__global__ __launch_bounds__(kThreads) void k_route(Args a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (t >= a.T) return;
    int key[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int e = lane + 64 * j;
        key[j] = e < a.E ? order_of(logit(a.z, kBf16, t * a.ld + e)) : kGone;
    }
    int top = key[0];
#pragma unroll
    for (int j = 1; j < kV; ++j) top = key[j] > top ? key[j] : top;
    const float m = value_of(wave_max(top));
    float total = 0.0f;
    if (!a.renorm) {
#pragma unroll
        for (int j = 0; j < kV; ++j)
            total += key[j] == kGone ? 0.0f : term(value_of(key[j]), m);
        total = wave_sum(total);
    }
    int id = 0;                              // lane i: the i-th expert and its term
    float mine = 0.0f;
    for (int i = 0; i < a.topk; ++i) {
        int best = key[0];
#pragma unroll
        for (int j = 1; j < kV; ++j) best = key[j] > best ? key[j] : best;
        best = wave_max(best);
        int e = kMaxE;
#pragma unroll
        for (int j = kV - 1; j >= 0; --j) {
            const uint64_t at = __ballot(key[j] == best);
            if (at) e = 64 * j + __builtin_ctzll(at);
        }
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (lane + 64 * j == e) key[j] = kGone;
        const float p = term(value_of(best), m);
        if (a.renorm) total += p;
        if (lane == i) {
            id = e;
            mine = p;
        }
    }
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = id;
        a.w[t * a.topk + lane] = total == 0.0f ? 0.0f : mine / total;
    }
}

template <int kBf16, int kV>
__global__ __launch_bounds__(kThreads) void k_route_grad(Args a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (t >= a.T) return;
    int id = -1;
    float w = 0.0f, gw = 0.0f;
    if (lane < a.topk) {
        id = a.ids[t * a.topk + lane];
        if (id >= 0 && id < a.E) {
            w = a.w[t * a.topk + lane];
            gw = a.g[t * a.topk + lane] * w;
        } else {
            id = -1;
        }
    }
    const float sum = wave_sum(gw);
    const float add = a.renorm ? gw - w * sum : gw;
    float d[kV];
    if (a.renorm) {
#pragma unroll
        for (int j = 0; j < kV; ++j) d[j] = 0.0f;
    } else {
        float z[kV], m = -INFINITY, total = 0.0f;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int e = lane + 64 * j;
            z[j] = e < a.E ? logit(a.z, kBf16, t * a.ld + e) : -INFINITY;
            m = fmaxf(m, z[j]);
        }
#pragma unroll
        for (int off = 32; off; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            z[j] = term(z[j], m);
            total += z[j];
        }
        total = wave_sum(total);
        const float by = total == 0.0f ? 0.0f : -sum / total;
#pragma unroll
        for (int j = 0; j < kV; ++j) d[j] = z[j] * by;
    }
    for (int i = 0; i < a.topk; ++i) {
        const int e = __shfl(id, i, 64);
        const float v = __shfl(add, i, 64);
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (lane + 64 * j == e) d[j] += v;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int e = lane + 64 * j;
        if (e < a.E) {
            if (kBf16) ((uint16_t*)a.dz)[t * a.E + e] = (uint16_t)bf16_bits(d[j], 0.0f);
            else ((float*)a.dz)[t * a.E + e] = d[j];
        }
    }
}

template <int kBf16, int kV>
void launch(const Args& a, bool grad, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + kThreads / 64 - 1) / (kThreads / 64)));
    if (grad) hipLaunchKernelGGL((k_route_grad<kBf16, kV>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_route<kBf16, kV>), grid, dim3(kThreads), 0, s, a);
}
template <int kBf16>
void launch(const Args& a, bool grad, hipStream_t s) {
    const int v = (a.E + 63) / 64;
    if (v <= 1) launch<kBf16, 1>(a, grad, s);
    else if (v <= 2) launch<kBf16, 2>(a, grad, s);
    else if (v <= 4) launch<kBf16, 4>(a, grad, s);
    else if (v <= 8) launch<kBf16, 8>(a, grad, s);
    else if (v <= 16) launch<kBf16, 16>(a, grad, s);
    else launch<kBf16, 64>(a, grad, s);
}

inline int check(int dtype, int64_t T, int32_t E, int64_t ld, int32_t topk, int renorm) {
    if (T < 0 || T >= ((int64_t)1 << 24) || E < 1 || E > kMaxE || ld < E || ld >= kMaxStride ||
        topk < 1 || topk > E || topk > kMaxTopk)
        return QUADS_ESHAPE;
    return ok_type(dtype) && (renorm == 0 || renorm == 1) ? QUADS_OK : QUADS_EINVAL;
}

}  // namespace routing
}  // namespace quads

using namespace quads;

extern "C" int quads_moe_route(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld,
                               int32_t topk, int renorm, int32_t* topk_ids, float* topk_w,
                               void* stream) {
    using namespace routing;
    if (int e = check(dtype, T, E, ld, topk, renorm)) return e;
    if (T == 0) return QUADS_OK;
    if (!ok_ptr(logits) || !ok_ptr4(topk_ids) || !ok_ptr4(topk_w)) return QUADS_EINVAL;
    const Args a = {logits, topk_ids, topk_w, nullptr, nullptr, T, ld, E, topk, renorm};
    if (dtype == QUADS_OUT_BF16) launch<1>(a, false, (hipStream_t)stream);
    else launch<0>(a, false, (hipStream_t)stream);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

extern "C" int quads_moe_route_backward(const void* logits, int dtype, int64_t T, int32_t E,
                                        int64_t ld, const int32_t* topk_ids, const float* topk_w,
                                        const float* g, int32_t topk, int renorm, void* dlogits,
                                        void* stream) {
    using namespace routing;
    if (int e = check(dtype, T, E, ld, topk, renorm)) return e;
    if (T == 0) return QUADS_OK;
    if ((!renorm && !ok_ptr(logits)) || !ok_ptr4(topk_ids) || !ok_ptr4(topk_w) || !ok_ptr4(g) ||
        !ok_ptr(dlogits) || (dlogits == logits && ld != E))
        return QUADS_EINVAL;
    const Args a = {logits, const_cast<int32_t*>(topk_ids), const_cast<float*>(topk_w), g, dlogits,
                    T, ld, E, topk, renorm};
    if (dtype == QUADS_OUT_BF16) launch<1>(a, true, (hipStream_t)stream);
    else launch<0>(a, true, (hipStream_t)stream);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}
