// Routing: the topk experts with the largest logits of each token, their weights,
// and the weights' gradient.
//
//   p = softmax(z),  w_i = p_{id_i}, or that divided by the sum over the topk
//   renorm 0: dz_v = a_i [v = id_i] - p_v A,   a_i = g_i w_i, A = sum a_i
//   renorm 1: dz_v = a_i - w_i A at v = id_i
//
// kL lanes (8 .. 64) share a token, kV neighbouring logits in the registers of each.  The
// order is by one unsigned number per logit, larger for a larger one: a float's bits, all
// turned over where it is negative, the sign alone where it is not.  topk times the lanes
// take their largest number, and the lowest lane that has it removes its first such logit.
// What bounds it is that chain of topk steps, about 50 operations each, not its bytes.
#include "block.h"

namespace quads {
namespace routing {

using namespace block;

constexpr int kMaxE = 4096, kMaxTopk = 64;
// Rows of many logits take a work-group of one wave: its shared memory holds them.
constexpr int threads_of(int v) { return v > 16 ? 64 : 256; }

struct Args {
    const void* z;
    int32_t* ids;
    float* w;
    const float* g;
    void* dz;
    int64_t T, ld;
    int E, topk, renorm;
};

// 0 is below every logit's number: a masked one's (-inf) is 0x007FFFFF.  z + 0 makes -0 a
// 0; a NaN of either sign stands above everything.
__device__ __forceinline__ uint32_t order_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    return z != z ? 0xFFFFFFFFu : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// exp(z - m), 0 for a masked logit even where nothing else is left.
__device__ __forceinline__ float term(float z, float m) {
    return z == -INFINITY ? 0.0f : expf(z - m);
}
// The logits kV * lane .. of a token; -inf behind the last.
template <int kBf16, int kV>
__device__ __forceinline__ void load_logits(const Args& a, int64_t t, int lane, float* z) {
    const void* row = row_at<kBf16>(a.z, t * a.ld);
#pragma unroll
    for (int j = 0; j < kV; j += kPer) {
        const int e = kV * lane + j;
        Raw<kBf16> r = {};
        if (t < a.T && e < a.E) r = load<kBf16>(row, e, a.E - e);
#pragma unroll
        for (int i = 0; i < kPer; ++i) z[j + i] = e + i < a.E ? r.get(i) : -INFINITY;
    }
}

template <int kBf16, int kL, int kV>
__global__ __launch_bounds__(threads_of(kV)) void k_route(Args a) {
    constexpr int kTokens = threads_of(kV) / kL;
    __shared__ uint2 s_top[kTokens][kMaxTopk];               // (id, number), in order
    const int token = threadIdx.x / kL, lane = threadIdx.x % kL;
    const int64_t t = (int64_t)blockIdx.x * kTokens + token;
    float z[kV];
    uint32_t key[kV];
    load_logits<kBf16, kV>(a, t, lane, z);
#pragma unroll
    for (int j = 0; j < kV; ++j) key[j] = kV * lane + j < a.E ? order_of(z[j]) : 0u;
    float m = 0.0f, total = 0.0f;
    for (int i = 0; i < a.topk; ++i) {
        uint32_t mine = key[0];
#pragma unroll
        for (int j = 1; j < kV; ++j) mine = larger(mine, key[j]);
        const uint32_t best = lanes_max<kL>(mine);
        if (i == 0) {
            m = value_of(best);
            if (!a.renorm) {
#pragma unroll
                for (int j = 0; j < kV; ++j) total += term(z[j], m);
                total = lanes_sum<kL>(total);
            }
        }
        const uint64_t at = __ballot(mine == best) >> ((threadIdx.x & 63) - lane);
        const bool have = (int)__builtin_ctzll(at) == lane;  // the token's lowest such lane
        int e = kV;
#pragma unroll
        for (int j = kV - 1; j >= 0; --j) e = key[j] == best ? j : e;
        if (have) s_top[token][i] = make_uint2((uint32_t)(kV * lane + e), best);
#pragma unroll
        for (int j = 0; j < kV; ++j) key[j] = have && j == e ? 0u : key[j];
    }
    __syncthreads();
    if (a.renorm) {
        for (int i = lane; i < a.topk; i += kL) total += term(value_of(s_top[token][i].y), m);
        total = lanes_sum<kL>(total);
    }
    if (t >= a.T) return;
    for (int i = lane; i < a.topk; i += kL) {
        const uint2 c = s_top[token][i];
        a.ids[t * a.topk + i] = (int32_t)c.x;
        a.w[t * a.topk + i] = total == 0.0f ? 0.0f : term(value_of(c.y), m) / total;
    }
}

// What the slots add goes through shared memory: the first slot of an id has the sum over
// all of its slots, in order, and puts it at the id's place (comparing every id with each
// of a lane's logits instead: 65536 x 128, top 8, 16.6 us against 14.9;
// 4096 x 4096 fp32 55 / 48).
template <int kBf16, int kL, int kV>
__global__ __launch_bounds__(threads_of(kV)) void k_route_grad(Args a) {
    constexpr int kTokens = threads_of(kV) / kL;
    __shared__ uint2 s_slot[kTokens][kMaxTopk];              // (id, a), in order
    __shared__ float s_add[kTokens][kL * kV];
    const int token = threadIdx.x / kL, lane = threadIdx.x % kL;
    const int64_t t = (int64_t)blockIdx.x * kTokens + token;
    float z[kV];
    if (!a.renorm) load_logits<kBf16, kV>(a, t, lane, z);
    float sum = 0.0f;
    for (int i = lane; i < a.topk; i += kL) {
        int id = -1;
        float gw = 0.0f;
        if (t < a.T) {
            id = a.ids[t * a.topk + i];
            if (id >= 0 && id < a.E) gw = a.g[t * a.topk + i] * a.w[t * a.topk + i];
            else id = -1;
        }
        s_slot[token][i] = make_uint2((uint32_t)id, __float_as_uint(gw));
        sum += gw;
    }
    sum = lanes_sum<kL>(sum);
#pragma unroll
    for (int j = 0; j < kV; ++j) s_add[token][kV * lane + j] = 0.0f;
    if (a.renorm) {
#pragma unroll
        for (int j = 0; j < kV; ++j) z[j] = 0.0f;
        for (int i = lane; i < a.topk; i += kL) {
            uint2& c = s_slot[token][i];
            if ((int)c.x >= 0)
                c.y = __float_as_uint(__uint_as_float(c.y) - a.w[t * a.topk + i] * sum);
        }
    } else {
        float m = z[0], total = 0.0f;
#pragma unroll
        for (int j = 1; j < kV; ++j) m = fmaxf(m, z[j]);
        m = value_of(lanes_max<kL>(order_of(m)));
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            z[j] = term(z[j], m);
            total += z[j];
        }
        total = lanes_sum<kL>(total);
        const float by = total == 0.0f ? 0.0f : -sum / total;
#pragma unroll
        for (int j = 0; j < kV; ++j) z[j] *= by;
    }
    __syncthreads();
    for (int i = lane; i < a.topk; i += kL) {
        const uint32_t id = s_slot[token][i].x;
        float v = 0.0f;
        bool first = (int)id >= 0;
        for (int k = 0; k < a.topk; ++k) {
            const uint2 c = s_slot[token][k];
            v += c.x == id ? __uint_as_float(c.y) : 0.0f;
            first = first && (c.x != id || k >= i);
        }
        if (first) s_add[token][id] = v;
    }
    __syncthreads();
    if (t >= a.T) return;
    void* row = row_at<kBf16>(a.dz, t * a.E);
#pragma unroll
    for (int j = 0; j < kV; j += kPer) {
        const int e = kV * lane + j;
#pragma unroll
        for (int i = 0; i < kPer; ++i) z[j + i] += s_add[token][e + i];
        if (e < a.E) store<kBf16>(row, e, a.E - e, pack<kBf16>(z + j));
    }
}

template <int kBf16, int kL, int kV>
void launch(const Args& a, bool grad, hipStream_t s) {
    constexpr int kTokens = threads_of(kV) / kL;
    const dim3 grid((unsigned)((a.T + kTokens - 1) / kTokens)), block(threads_of(kV));
    if (grad) hipLaunchKernelGGL((k_route_grad<kBf16, kL, kV>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_route<kBf16, kL, kV>), grid, block, 0, s, a);
}
template <int kBf16>
void launch(const Args& a, bool grad, hipStream_t s) {
    if (a.E <= 64) launch<kBf16, 8, 8>(a, grad, s);
    else if (a.E <= 128) launch<kBf16, 16, 8>(a, grad, s);
    else if (a.E <= 256) launch<kBf16, 32, 8>(a, grad, s);
    else if (a.E <= 512) launch<kBf16, 64, 8>(a, grad, s);
    else if (a.E <= 1024) launch<kBf16, 64, 16>(a, grad, s);
    else launch<kBf16, 64, 64>(a, grad, s);
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
