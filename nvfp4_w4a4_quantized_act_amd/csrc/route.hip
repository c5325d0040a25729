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
// take their largest number, and the lane that has it removes it.  What bounds it is the
// vector units, 330 operations for eight steps of bf16 logits, not its bytes (65536 x 128,
// top 8, bf16 11.9 us, 1.8 TB/s; the gradient 13.8 us, 2.9 TB/s).
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
// What exponents are taken from: the largest logit, 0 where every one is masked (whose
// terms are then 0, as a masked logit's are).
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
// exp(z - m) three times.  A weight's numerator: expf (16 operations).
__device__ __forceinline__ float numerator(float z, float m) { return expf(z - m); }
// A term of the forward call's sum over all experts: the hardware's 2^x of a rounded product
// (3 operations), off by up to 1.5 * 2^-24 |z - m| of itself, which leaves the sum nothing
// to speak of (a term far below the largest is as much smaller).
__device__ __forceinline__ float term(float z, float m) {
    return __builtin_amdgcn_exp2f((z - m) * 1.44269504f);
}
// Every expert's probability in the gradient, where an unlikely one stands by itself: what
// the product's rounding and log2(e)'s leave out is put back (9 operations, 2 ulps; 0 below
// 2^-126).  65536 x 128 bf16 13.8 us, 14.4 by expf, 13.1 by `term`, which is off by 64 *
// 2^-24 in experts 80 below the largest.
__device__ __forceinline__ float probable(float z, float m) {
    const float d = z - m, h = d * 1.44269504f, e = __builtin_amdgcn_exp2f(h);
    const float left = fmaf(d, 1.92596299e-8f, fmaf(d, 1.44269504f, -h)) * 0.693147181f;
    return e == 0.0f ? 0.0f : fmaf(e, left, e);              // -inf has no product
}
// The logits kV * lane .. of a token; -inf behind the last.
template <int kBf16, int kV>
__device__ __forceinline__ void load_logits(const Args& a, int64_t t, int lane, float* z) {
    const void* row = row_at<kBf16>(a.z, t * a.ld);
    const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
    for (int j = 0; j < kV; j += kPer) {
        const int e = kV * lane + j;
        Raw<kBf16> r;
        for (int i = 0; i < (kBf16 ? 1 : 2); ++i) r.q[i] = words4{none, none, none, none};
        if (t < a.T && e < a.E) r = load<kBf16>(row, e, a.E - e);
#pragma unroll
        for (int i = 0; i < kPer; ++i) z[j + i] = r.get(i);
        if (e < a.E && a.E - e < kPer) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) z[j + i] = i < a.E - e ? z[j + i] : -INFINITY;
        }
    }
}

// Both values, not their places: a choice between two registers of an array becomes a
// search through it.
__device__ __forceinline__ uint32_t pick(bool c, uint32_t a, uint32_t b) { return c ? a : b; }
// A lane's eight numbers, the largest first (19 exchanges).
__device__ __forceinline__ void sort8(uint32_t* k) {
    constexpr int kPairs[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6},
                                   {5, 7}, {1, 2}, {5, 6}, {0, 4}, {1, 5}, {2, 6}, {3, 7},
                                   {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) {
        const uint32_t x = k[kPairs[i][0]], y = k[kPairs[i][1]];
        k[kPairs[i][0]] = larger(x, y);
        k[kPairs[i][1]] = x < y ? x : y;
    }
}

// The place of the first of eight numbers that is `best`; that one becomes 0 if `have`, and
// `most` the largest of them then.
__device__ __forceinline__ int take(bool have, uint32_t* k, uint32_t best, uint32_t& most) {
    int e = 8;
#pragma unroll
    for (int j = 7; j >= 0; --j) e = k[j] == best ? j : e;
    most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        k[j] = pick(have && j == e, 0u, k[j]);
        most = larger(most, k[j]);
    }
    return e;
}

// Up to 512 experts (kV 8) the numbers carry their place: a bf16 logit's 16 bits above the
// place's complement, an fp32 logit's upper bits above it.  They differ, larger ones and
// among equal ones lower places come first, and a step is the lanes' maximum and a lane's
// shift, about 16 operations where finding and removing the first equal number takes 50
// (in all 65536 x 128 bf16 11.9 us / 20, 16384 x 256 fp32 10.2 / 12.6).
// fp32 numbers that differ only in the bits below tell so by equal bits above: their wave
// takes the steps that compare all bits.  So does every wave beyond 512 experts, by the
// largest of eights, of which a step changes one (looking through all 64 numbers of a lane
// in each step 4096 x 4096 fp32, top 8, 51 us against 32, 64 x 4096 17 / 8).
template <int kBf16, int kL, int kV>
__global__ __launch_bounds__(threads_of(kV)) void k_route(Args a) {
    constexpr int kTokens = threads_of(kV) / kL;
    constexpr bool kPlaced = kV == 8, kWithValue = kPlaced && kBf16;
    constexpr uint32_t kPlace = kWithValue ? 0xFFFFu : kL * kV - 1;
    __shared__ uint32_t s_top[kTokens][kMaxTopk];            // kPlace - place in the lower bits
    __shared__ __align__(16) float s_z[kWithValue ? 1 : kTokens][kWithValue ? 4 : kL * kV];
    const int token = threadIdx.x / kL, lane = threadIdx.x % kL;
    const int64_t t = (int64_t)blockIdx.x * kTokens + token;
    float z[kV];
    uint32_t key[kV];
    load_logits<kBf16, kV>(a, t, lane, z);
    // places behind the last expert are as masked ones, and stand behind those
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        key[j] = order_of(z[j]);
        most = larger(most, key[j]);
    }
    const float m = base_of(value_of(lanes_max<kL>(most)));
    if (!kWithValue) {
#pragma unroll
        for (int j = 0; j < kV; j += 4)
            *reinterpret_cast<float4*>(&s_z[token][kV * lane + j]) =
                make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]);
    }
    float total = 0.0f;
    if (!a.renorm) {
#pragma unroll
        for (int j = 0; j < kV; ++j) total += term(z[j], m);
        total = lanes_sum<kL>(total);
    }
    bool whole = !kPlaced;                                   // compare all bits
    if constexpr (kPlaced) {
        const uint32_t place = kPlace - (uint32_t)(kV * lane);
        uint32_t k[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) k[j] = (key[j] & ~kPlace) | (place - j);
        sort8(k);
        uint32_t before = 0;
        for (int i = 0; i < a.topk; ++i) {
            const uint32_t best = lanes_max<kL>(k[0]);
            if (lane == 0) s_top[token][i] = best;
            if (!kBf16) whole = whole || ((best ^ before) & ~kPlace) == 0;
            before = best;
            const bool have = k[0] == best;
#pragma unroll
            for (int j = 0; j + 1 < kV; ++j) k[j] = pick(have, k[j + 1], k[j]);
            k[kV - 1] = pick(have, 0u, k[kV - 1]);
        }
        if (!kBf16) {                                        // the next one decides nothing?
            const uint32_t next = lanes_max<kL>(k[0]);
            whole = whole || ((next ^ before) & ~kPlace) == 0;
        }
    }
    if constexpr (kPlaced && !kBf16) {
        if (__ballot(whole)) {
            for (int i = 0; i < a.topk; ++i) {
                uint32_t mine = key[0];
#pragma unroll
                for (int j = 1; j < kV; ++j) mine = larger(mine, key[j]);
                const uint32_t best = lanes_max<kL>(mine);
                const uint64_t at = __ballot(mine == best) >> ((threadIdx.x & 63) - lane);
                const bool have = (int)__builtin_ctzll(at) == lane;  // the token's lowest such lane
                const int e = take(have, key, best, mine);
                if (have) s_top[token][i] = kPlace - (uint32_t)(kV * lane + e);
            }
        }
    }
    if constexpr (!kPlaced) {                                // a wave is one token's
        constexpr int kParts = kV / 8;
        uint32_t part[kParts];                               // the largest of eight numbers
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
            part[q] = key[8 * q];
#pragma unroll
            for (int j = 1; j < 8; ++j) part[q] = larger(part[q], key[8 * q + j]);
        }
        for (int i = 0; i < a.topk; ++i) {
            uint32_t mine = part[0];
#pragma unroll
            for (int q = 1; q < kParts; ++q) mine = larger(mine, part[q]);
            const uint32_t best = lanes_max<kL>(mine);
            const int winner = __builtin_ctzll(__ballot(mine == best));
            int in = 0;
#pragma unroll
            for (int q = kParts - 1; q >= 0; --q) in = part[q] == best ? q : in;
            in = __builtin_amdgcn_readlane(in, winner);
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                if (q != in) continue;
                const int e = take(lane == winner, key + 8 * q, best, part[q]);
                if (lane == winner) s_top[token][i] = kPlace - (uint32_t)(kV * lane + 8 * q + e);
            }
        }
    }
    __syncthreads();
    auto chosen = [&](int i) {                               // its numerator
        const uint32_t c = s_top[token][i];
        if (kWithValue) return numerator(value_of((int)c < 0 ? c & ~kPlace : c | kPlace), m);
        return numerator(s_z[kWithValue ? 0 : token][kPlace - (c & kPlace)], m);
    };
    if (a.renorm) {
        for (int i = lane; i < a.topk; i += kL) total += chosen(i);
        total = lanes_sum<kL>(total);
    }
    if (t >= a.T) return;
    for (int i = lane; i < a.topk; i += kL) {
        a.ids[t * a.topk + i] = (int32_t)(kPlace - (s_top[token][i] & kPlace));
        a.w[t * a.topk + i] = total == 0.0f ? 0.0f : chosen(i) / total;
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
        m = base_of(value_of(lanes_max<kL>(order_of(m))));
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            z[j] = probable(z[j], m);
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
