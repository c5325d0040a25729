// Log-probabilities of given tokens, entropy and top alternatives, and their
// gradient (include/quads_head.h).
//
// Forward.  With d = it (z - m) the log-sum s = ln sum e^d and the entropy
// H = s - (sum e^d d) / sum e^d come from one pass over the row: every thread
// keeps a running maximum with the two sums, rescaled when the maximum rises,
// and the threads' statistics are joined at the end.  The top alternatives
// come from the same pass (k_logprob below).  A row is one work-group's where
// there are rows enough; else it is split into parts whose results k_merge
// joins.  Everything is summed in a fixed order.
//
// Backward: dz = it (g_lp 1[v = id] - p (g_lp + g_H (ln p + H))), one read and
// one write of the row, the token's entry patched by the thread that holds it.
#include "logits.h"

namespace quads {
namespace head {

// ------------------------------------------------------------ alternatives --

// Ranks by value (signed zeros equal), then by lower index; never 0.
__device__ __forceinline__ uint32_t value_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t rank_key(float z, uint32_t v) {
    return ((uint64_t)value_key(z) << 32) | (0xFFFFFFFFu - v);
}
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t b = (uint32_t)(k >> 32);
    return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

constexpr int kCand = 1024;                    // candidates kept at once

struct __align__(16) Cand {
    uint64_t key[kCand + 8];
    uint16_t top[2][kThreads];                 // upper halves of the threads' maxima's keys
    int n;
};

// The smallest fp32 above x (x no NaN; NaN above +inf, which no entry reaches).
__device__ __forceinline__ float next_up(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return __uint_as_float((int32_t)b >= 0 ? b + 1u : b - 1u);
}

// The k-th largest of the wave's values h (halves of keys, kPerLane a lane), 0
// if there are fewer: one bit at a time, counted with ballots.
template <int kPerLane>
__device__ __forceinline__ uint32_t kth_half(const uint32_t* h, int k) {
    uint32_t t = 0;
#pragma unroll
    for (int b = 15; b >= 0; --b) {
        const uint32_t x = t | (1u << b);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) n += __popcll(__ballot(h[i] >= x));
        if (n >= k) t = x;
    }
    return t;
}

// The lowest value of a half (none below -inf).
__device__ __forceinline__ float half_bound(uint32_t t) {
    return t <= 0x007Fu ? -INFINITY : key_value((uint64_t)(t << 16) << 32);
}
// A value that at least k of the work-group's values (key halves in `top`)
// reach: the k-th largest half, rounded down.  Every wave finds it by itself.
__device__ __forceinline__ float kth_bound(const uint16_t* top, int k) {
    const uint2 w = reinterpret_cast<const uint2*>(top)[threadIdx.x & 63];
    const uint32_t h[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
    return half_bound(kth_half<4>(h, k));
}
// The same from one wave's values in registers.
__device__ __forceinline__ float kth_bound(const float (&m)[4], int k) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = value_key(m[i]) >> 16;
    return half_bound(kth_half<4>(h, k));
}

// A thread's maximum, or that of kThr / kThreads neighbours, into `top`.
template <int kThr>
__device__ __forceinline__ void set_top(uint16_t* top, float m) {
    constexpr int kOf = kThr / kThreads;
    static_assert(kOf == 1 || kOf == 4, "one thread's or four neighbours' maximum");
    if (kOf == 4) {
        m = fmaxf(m, dpp_move<0xB1, 0xF>(m, m));           // quad_perm:[1,0,3,2]
        m = fmaxf(m, dpp_move<0x4E, 0xF>(m, m));           // quad_perm:[2,3,0,1]
    }
    if (threadIdx.x % kOf == 0) top[threadIdx.x / kOf] = (uint16_t)(value_key(m) >> 16);
}

// Drops the candidates whose half is below the k-th largest one.
template <int kPerLane>
__device__ __forceinline__ uint64_t kth_key(const Cand& c, int n, int k) {
    uint32_t h[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int at = (int)(threadIdx.x & 63) + 64 * i;
        h[i] = at < n ? (uint32_t)(c.key[at] >> 48) : 0;
    }
    return (uint64_t)kth_half<kPerLane>(h, k) << 48;
}
template <int kThr>
__device__ __forceinline__ int drop_low(Cand& c, int n, int k) {
    uint64_t mine[kCand / kThr];
    __syncthreads();
    const uint64_t low = n <= 256 ? kth_key<4>(c, n, k) : kth_key<kCand / 64>(c, n, k);
#pragma unroll
    for (int i = 0; i < kCand / kThr; ++i) {
        const int at = threadIdx.x + i * kThr;
        mine[i] = at < n ? c.key[at] : 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) c.n = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCand / kThr; ++i)
        if (mine[i] >= low && mine[i] != 0) c.key[atomicAdd(&c.n, 1)] = mine[i];
    __syncthreads();
    return c.n;
}

// Sorts the n candidates and keeps the k largest (c.n is set; barriers on
// both sides).  Each entry's place is the number of larger ones, eight read
// at a time; candidates well beyond k are dropped before.
template <int kThr>
__device__ __forceinline__ void keep_top(Cand& c, int n, int k) {
    if (n > k + k / 2 + 16) n = drop_low<kThr>(c, n, k);
    uint64_t mine[kCand / kThr];
    int place[kCand / kThr];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCand / kThr; ++i) {
        const int at = threadIdx.x + i * kThr;
        mine[i] = at < n ? c.key[at] : 0;
        place[i] = 0;
    }
    if (threadIdx.x < 8) c.key[n + threadIdx.x] = 0;       // smaller than any
    __syncthreads();
    for (int j = 0; j < n; j += 8) {
        uint64_t x[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) x[b] = c.key[j + b];
#pragma unroll
        for (int b = 0; b < 8; ++b) place[0] += x[b] > mine[0] ? 1 : 0;
        if (n > kThr) {
#pragma unroll
            for (int i = 1; i < kCand / kThr; ++i)
                if (kThr >= 256 || i * kThr < n) {
#pragma unroll
                    for (int b = 0; b < 8; ++b) place[i] += x[b] > mine[i] ? 1 : 0;
                }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCand / kThr; ++i)
        if (mine[i] != 0 && place[i] < k) c.key[place[i]] = mine[i];
    if (threadIdx.x == 0) c.n = n < k ? n : k;
    __syncthreads();
}

// ----------------------------------------------------------------- forward --

struct Out {
    const int32_t* ids;
    float it;
    int topk;
    float *logp, *entropy, *stats, *top_logp;
    int32_t* top_id;
};

// What the parts of a row leave for k_merge: per part its statistics and, in
// a second array, its topk candidates in order (0: none).
struct Parts {
    float4* stat;
    uint64_t* key;
};

// The row's token, read early.
struct Token {
    int id;
    float z;
};
template <int kBf16>
__device__ __forceinline__ Token load_token(const Out& o, const Row<kBf16>& r, int64_t t) {
    Token k = {-1, 0.0f};
    if (o.ids && threadIdx.x == 0) {
        k.id = o.ids[t];
        if (k.id >= 0 && k.id < r.V) k.z = r.entry(k.id);
    }
    return k;
}

// The outputs of row t from its statistics and its n largest entries (thread
// 0, and all for the alternatives; key in LDS, sorted).  n < topk: no further entry is
// above -inf, so that the masked ones of lowest index follow.
template <int kBf16>
__device__ __forceinline__ void finish(const Out& o, const Row<kBf16>& r, int64_t t, const Stat& a,
                                       const Token& k, uint64_t* key, int n) {
    const double ls = log_sum(a);
    if (threadIdx.x == 0) {
        o.stats[2 * t] = a.m;
        o.stats[2 * t + 1] = (float)ls;
        if (o.entropy)
            o.entropy[t] = a.m == -INFINITY && a.s == 0.0f
                               ? 0.0f
                               : (float)(ls - 0.69314718055994531 * (double)a.u / (double)a.s);
        if (o.ids)
            o.logp[t] = k.id >= 0 && k.id < r.V ? (float)ln_p(k.z, a.m, ls, o.it) : 0.0f;
    }
    if (o.topk == 0) return;
    const bool number = ls == ls;              // no NaN or +inf in the row
    if (n < o.topk && number) {
        if (threadIdx.x < 64) {
            for (int b = 0; b < r.V && n < o.topk; b += 64) {
                const int v = b + (int)threadIdx.x;
                const bool masked = v < r.V && r.entry(v) == -INFINITY;
                const uint64_t all = __ballot(masked);
                const int at = n + __popcll(all & ((1ull << threadIdx.x) - 1ull));
                if (masked && at < o.topk) key[at] = rank_key(-INFINITY, (uint32_t)v);
                n += __popcll(all);
            }
        }
        __syncthreads();
        n = o.topk;
    }
    for (int i = threadIdx.x; i < o.topk; i += blockDim.x) {
        const int64_t at = t * o.topk + i;
        const bool have = n >= o.topk;         // else any indices
        o.top_id[at] = have ? key_index(key[i]) : i;
        o.top_logp[at] = have ? (float)ln_p(key_value(key[i]), a.m, ls, o.it) : NAN;
    }
}

// One work-group: part blockIdx.x % parts of row blockIdx.x / parts, in chunks
// of kVecs vectors per thread, the next chunk's vectors requested before the
// present one is worked on.
//
// kTop: a candidate is an entry above a value that topk earlier entries reach
// (and above -inf).  That bound is the topk-th largest of the threads' running
// maxima, taken after the first chunk and again after 2, 4, 8, ... chunks
// (entries of the first chunk count from the bound on, later ones only above
// it, as their indices are higher), so that a random row yields about topk (1
// + log2 of the chunks) candidates and most vectors are compared with one
// number (256 maxima: one a thread, one of four threads in a wide work-group,
// four a thread, in registers, in a single wave).  The candidates are sorted
// once, at the end.  Where there were more
// than there is room for (equal or rising entries) the part is read again,
// up to 256 entries at a time, the candidates cut to the topk largest in between.
template <int kBf16, bool kEntropy, bool kTop, int kVecs, int kThr = kThreads>
__global__ __launch_bounds__(kThr) void k_logprob(const void* z, int64_t V, int64_t ld, int parts,
                                                  Out o, Parts p) {
    constexpr int kPer = Row<kBf16>::kPer;
    constexpr int kChunk = kThr * kVecs;
    constexpr bool kOneWave = kThr == 64;
    constexpr int kRead = kThr < kThreads ? kThr : kThreads;
    __shared__ Stat s_stat[kThr / 64];
    __shared__ __align__(16) char s_cand[kTop ? sizeof(Cand) : 16];
    Cand& c = *reinterpret_cast<Cand*>(s_cand);
    const int64_t t = blockIdx.x / (unsigned)parts;
    const int part = (int)(blockIdx.x % (unsigned)parts);
    const Row<kBf16> r(z, t, ld, V);
    const float cl = o.it * kLog2e;
    const int chunks = (r.nvec + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * part / parts);
    const int c1 = (int)((int64_t)chunks * (part + 1) / parts);
    const int topk = o.topk;

    auto load = [&](uint4 (&q)[kVecs], int ch) {
        if (ch >= c1) return;
        const int j0 = ch * kChunk;
        if (r.whole(j0) && r.whole(j0 + kChunk - 1)) {
            const uint4* a = r.vec(j0 + threadIdx.x);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) q[i] = a[i * kThr];
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int j = j0 + i * kThr + threadIdx.x;
                if (r.whole(j)) q[i] = *r.vec(j);
                else q[i] = r.part(j);
            }
        }
    };

    uint4 q[kVecs], next[kVecs];
    load(next, c0);
    const Token token = parts == 1 ? load_token<kBf16>(o, r, t) : Token{-1, 0.0f};
    Stat a = {-INFINITY, 0.0f, 0.0f};
    float bound = -INFINITY;                   // candidates reach it
    int fresh = 0;
    float most[kVecs];                         // one wave: maxima of its vectors
#pragma unroll
    for (int i = 0; i < kVecs; ++i) most[i] = -INFINITY;
    if (kTop) {
        if (threadIdx.x == 0) c.n = 0;
        __syncthreads();
    }
    for (int ch = c0; ch < c1; ++ch) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) q[i] = next[i];
        load(next, ch + 1);
        float vm[kVecs], m = a.m;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            vm[i] = get<kBf16>(q[i], 0);
#pragma unroll
            for (int e = 1; e < kPer; ++e) vm[i] = fmaxf(vm[i], get<kBf16>(q[i], e));
            m = fmaxf(m, vm[i]);
        }
        stat_raise(a, m, cl);
        const float base = stat_base(m);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const float d = (get<kBf16>(q[i], e) - base) * cl;
                const float x = __builtin_amdgcn_exp2f(d);
                a.s += x;
                if (kEntropy) a.u = __builtin_fmaf(x, fmaxf(d, kNoTerm), a.u);
            }
        if (kTop) {
            const int nth = ch - c0;
            if constexpr (kOneWave) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) most[i] = fmaxf(most[i], vm[i]);
                if (nth == 0) bound = kth_bound(most, topk);
            } else if (nth == 0) {
                set_top<kThr>(c.top[0], m);
                __syncthreads();
                bound = kth_bound(c.top[0], topk);
            }
            const float reach = fmaxf(bound, next_up(-INFINITY));
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (vm[i] >= reach) {
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const float x = get<kBf16>(q[i], e);
                        if (x >= reach) {
                            const int at = atomicAdd(&c.n, 1);
                            const int v = r.index(ch * kChunk + i * kThr + threadIdx.x, e);
                            if (at < kCand) c.key[at] = rank_key(x, (uint32_t)v);
                        }
                    }
                }
            if (nth == 0) {
                bound = next_up(bound);
            } else if ((nth & (nth + 1)) == 0 && ch + 1 < c1) {
                // (two sets of maxima in turn: a wave writes the second next
                // one only after all have read this one)
                if constexpr (kOneWave) {
                    bound = fmaxf(bound, next_up(kth_bound(most, topk)));
                } else {
                    fresh ^= 1;
                    set_top<kThr>(c.top[fresh], m);
                    __syncthreads();
                    bound = fmaxf(bound, next_up(kth_bound(c.top[fresh], topk)));
                }
            }
        }
    }

    a = group_stat<kThr / 64>(a, cl, s_stat);
    int n = 0;
    if (kTop) {
        n = c.n;                               // (group_stat has a barrier)
        if (n > kCand) {
            __syncthreads();
            n = 0;
            if (threadIdx.x == 0) c.n = 0;
            __syncthreads();
            uint64_t over = 0;                 // the topk-th candidate, once cut
            const int v0 = max(r.index(c0 * kChunk, 0), 0);
            const int v1 = min((int64_t)r.V, (int64_t)c1 * kChunk * kPer - r.shift);
            for (int v = v0; v < v1; v += kRead * 8) {
                uint64_t k[8];
                bool any = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = v + i * kRead + (int)threadIdx.x;
                    const bool mine = kThr == kRead || threadIdx.x < kRead;
                    const float x = mine && at < v1 ? r.entry(at) : -INFINITY;
                    k[i] = x > -INFINITY ? rank_key(x, (uint32_t)at) : 0;
                    any = any || k[i] > over;
                }
                if (!__syncthreads_or(any)) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (n + kRead > kCand) {
                        keep_top<kThr>(c, n, topk);
                        over = c.n == topk ? c.key[topk - 1] : 0;
                        __syncthreads();
                    }
                    if (k[i] > over) c.key[atomicAdd(&c.n, 1)] = k[i];
                    __syncthreads();
                    n = c.n;
                    __syncthreads();
                }
            }
        }
        keep_top<kThr>(c, n, topk);
        n = c.n;
    }
    if (parts == 1) {
        finish<kBf16>(o, r, t, a, token, c.key, n);
    } else {
        if (threadIdx.x == 0) p.stat[blockIdx.x] = make_float4(a.m, a.s, a.u, 0.0f);
        if (kTop && (int)threadIdx.x < topk)
            p.key[(int64_t)blockIdx.x * topk + threadIdx.x] =
                (int)threadIdx.x < n ? c.key[threadIdx.x] : 0;
    }
}

// Joins the parts of a row.  The statistics: lane l of every wave holds part
// l (kMaxParts = 64).  The alternatives: the parts' candidates at or above
// the topk-th largest of the threads' maxima, sorted; all of them, cut in
// between, if those are more than there is room for.
template <int kBf16>
__global__ __launch_bounds__(kThreads) void k_merge(const void* z, int64_t V, int64_t ld,
                                                    int parts, Out o, Parts p) {
    __shared__ Cand c;
    const int64_t t = blockIdx.x;
    const Row<kBf16> r(z, t, ld, V);
    const int lane = threadIdx.x & 63;
    const Token token = load_token<kBf16>(o, r, t);
    Stat a = {-INFINITY, 0.0f, 0.0f};
    if (lane < parts) {
        const float4 q = p.stat[t * parts + lane];
        a = {q.x, q.y, q.z};
    }
    int n = 0;
    if (o.topk > 0) {
        const uint64_t* key = p.key + t * parts * o.topk;
        const int all = parts * o.topk;
        uint64_t most = 0;
        for (int i = threadIdx.x; i < all; i += kThreads) most = key[i] > most ? key[i] : most;
        c.top[0][threadIdx.x] = (uint16_t)(most >> 48);
        if (threadIdx.x == 0) c.n = 0;
        __syncthreads();
        const uint64_t low = (uint64_t)value_key(kth_bound(c.top[0], o.topk)) << 32;
        for (int i = threadIdx.x; i < all; i += kThreads) {
            const uint64_t k = key[i];
            if (k > low) {                     // (a key's index half is not 0)
                const int at = atomicAdd(&c.n, 1);
                if (at < kCand) c.key[at] = k;
            }
        }
        __syncthreads();
        n = c.n;
        if (n > kCand) {
            __syncthreads();
            n = 0;
            if (threadIdx.x == 0) c.n = 0;
            __syncthreads();
            uint64_t over = 0;
            for (int b = 0; b < all; b += kThreads) {
                if (n + kThreads > kCand) {
                    keep_top<kThreads>(c, n, o.topk);
                    over = c.n == o.topk ? c.key[o.topk - 1] : 0;
                    __syncthreads();
                }
                const int i = b + threadIdx.x;
                const uint64_t k = i < all ? key[i] : 0;
                if (k > over) c.key[atomicAdd(&c.n, 1)] = k;
                __syncthreads();
                n = c.n;
                __syncthreads();
            }
        }
        keep_top<kThreads>(c, n, o.topk);
        n = c.n;
    }
    a = wave_stat(a, o.it * kLog2e);
    finish<kBf16>(o, r, t, a, token, c.key, n);
}

// ---------------------------------------------------------------- backward --

template <int kBf16>
__global__ __launch_bounds__(kThreads) void k_logprob_bwd(const void* z, int64_t V, int64_t ld,
                                                          int parts, const int32_t* ids, float it,
                                                          const float* stats,
                                                          const float* entropy,
                                                          const float* g_logp,
                                                          const float* g_entropy, void* dz) {
    constexpr int kPer = Row<kBf16>::kPer;
    // the last rows first: they are the ones the forward pass has left in the
    // cache (4096 x 65536 bf16, both passes: 327 -> 322 us)
    const unsigned at = gridDim.x - 1 - blockIdx.x;
    const int64_t t = at / (unsigned)parts;
    const int part = (int)(at % (unsigned)parts);
    const Row<kBf16> r(z, t, ld, V);
    char* out = (char*)dz + (r.at - (const char*)z);
    const int chunks = (r.nvec + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * part / parts);
    const int c1 = (int)((int64_t)chunks * (part + 1) / parts);

    const float m = stats[2 * t], ls = stats[2 * t + 1];
    const int id = ids ? ids[t] : -1;
    const bool have = id >= 0 && id < r.V;
    const float gl = g_logp && have ? it * g_logp[t] : 0.0f;
    const float gh = g_entropy ? it * g_entropy[t] : 0.0f;
    // with x = log2(p sum): dz = it g_lp 1[v = id] - 2^x (f0 + f1 x), both
    // factors by 1 / sum
    const float inv = recip_sum(ls);
    const float f0 = (g_entropy ? __builtin_fmaf(gh, entropy[t] - ls, gl) : gl) * inv;
    const float f1 = gh * kLn2 * inv;
    const bool none = m == -INFINITY && ls == ls;          // no unmasked entry: no gradient
    const float cl = it * kLog2e;
    const int idv = have ? (id + r.shift) / kPer : -1, ide = have ? (id + r.shift) % kPer : 0;

    for (int ch = c0; ch < c1; ++ch) {
        uint4 q[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = ch * kChunk + i * kThreads + threadIdx.x;
            if (none) q[i] = make_uint4(0, 0, 0, 0);
            else if (r.whole(j)) q[i] = *r.vec(j);
            else q[i] = r.part(j);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = ch * kChunk + i * kThreads + threadIdx.x;
            float g[8];
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const float x = (get<kBf16>(q[i], e) - m) * cl;
                g[e] = -__builtin_amdgcn_exp2f(x) * __builtin_fmaf(f1, fmaxf(x, kNoTerm), f0);
            }
            if (j == idv) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) g[e] += e == ide ? gl : 0.0f;
            }
            if (none) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) g[e] = 0.0f;
            }
            if (j < r.nvec) store_vec<kBf16>(r, out, j, put<kBf16>(g));
        }
    }
}

// Rows of one work-group each that leave the GPU half empty, too many for wide
// ones (wide_rows), and longer than two chunks wait for each chunk's loads:
// their sums take four times the vectors at once (in us, calls in turn, 4 / 16
// vectors: 400 x 30000 bf16 19.2 / 16.2; not for 800 x 30000 fp32 28.5 / 30.6).
constexpr int kVecsFew = 16;
// Vectors of a row that a wave takes alone (short_rows; in us, calls in turn
// from a graph, 256 / 64 threads; no alternatives: 4096 x 2000 fp32 13.9 / 9.9,
// 4096 x 300 bf16 18.1 / 8.2, not for 4096 x 4000 fp32 15.0 / 15.7; top 8: 4096 x
// 2000 fp32 23.6 / 17.2, 2048 x 2000 bf16 16.7 / 10.1; top 128: 4096 x 2000 fp32
// 34.8 / 31.3, not for 2048 rows 20.7 / 24.3).
constexpr int kShortSum = 512;
template <int kBf16>
inline bool few_rows(int64_t T, int64_t V, int parts) {
    return parts == 1 && T <= 512 && V > 2 * kChunk * (int64_t)Row<kBf16>::kPer;
}

template <int kBf16, bool kEntropy, bool kTop>
void launch_rows(const void* z, int64_t T, int64_t V, int64_t ld, int parts, const Out& o,
                 const Parts& p, hipStream_t st) {
    const dim3 grid((unsigned)(T * parts)), block(kThreads);
    if (short_rows(o.topk > 64 ? T / 2 : T,
                   row_vectors(V, kBf16 ? QUADS_OUT_BF16 : QUADS_OUT_F32), kShortSum))
        hipLaunchKernelGGL((k_logprob<kBf16, kEntropy, kTop, kVecs, 64>), grid, dim3(64), 0, st, z,
                           V, ld, 1, o, p);
    else if (wide_rows<kBf16>(T, V, parts))
        hipLaunchKernelGGL((k_logprob<kBf16, kEntropy, kTop, kVecs, kWideThreads>), grid,
                           dim3(kWideThreads), 0, st, z, V, ld, 1, o, p);
    else if (few_rows<kBf16>(T, V, parts))
        hipLaunchKernelGGL((k_logprob<kBf16, kEntropy, kTop, kVecsFew>), grid, block, 0, st, z, V,
                           ld, parts, o, p);
    else
        hipLaunchKernelGGL((k_logprob<kBf16, kEntropy, kTop, kVecs>), grid, block, 0, st, z, V, ld,
                           parts, o, p);
}

template <int kBf16>
void launch_forward(const void* z, int64_t T, int64_t V, int64_t ld, int parts, const Out& o,
                    const Parts& p, hipStream_t st) {
    if (o.topk > 0 && o.entropy)
        launch_rows<kBf16, true, true>(z, T, V, ld, parts, o, p, st);
    else if (o.topk > 0)
        launch_rows<kBf16, false, true>(z, T, V, ld, parts, o, p, st);
    else if (o.entropy)
        launch_rows<kBf16, true, false>(z, T, V, ld, parts, o, p, st);
    else
        launch_rows<kBf16, false, false>(z, T, V, ld, parts, o, p, st);
    if (parts > 1)
        hipLaunchKernelGGL((k_merge<kBf16>), dim3((unsigned)T), dim3(kThreads), 0, st, z, V, ld,
                           parts, o, p);
}

}  // namespace head
}  // namespace quads

using namespace quads;

// Statistics and candidates of the parts, as many as either type is split into.
extern "C" size_t quads_token_logprob_ws(int64_t T, int64_t V, int32_t topk) {
    if (T < 1 || V < 1 || topk < 0) return 0;
    const int parts =
        head::row_parts(T, V, QUADS_OUT_F32, topk > 0 ? head::kWholeTop : head::kWhole);
    return parts > 1 ? (size_t)T * parts * (16 + 8 * (size_t)topk) : 0;
}

extern "C" int quads_token_logprob(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                   const int32_t* ids, float inv_temp, int32_t topk, float* logp,
                                   float* entropy, float* stats, float* top_logp, int32_t* top_id,
                                   void* ws, size_t ws_bytes, void* stream) {
    const int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc != QUADS_OK) return rc;
    if (topk < 0 || topk > QUADS_TOP_MAX || topk > V) return QUADS_ESHAPE;
    if (T == 0) return QUADS_OK;
    if (!head::ok_opt4(ids) || !head::ok_opt4(logp) || (ids == nullptr) != (logp == nullptr) ||
        !head::ok_opt4(entropy) || !ok_ptr4(stats))
        return QUADS_EINVAL;
    if (topk > 0 && (!ok_ptr4(top_logp) || !ok_ptr4(top_id))) return QUADS_EINVAL;
    const size_t need = quads_token_logprob_ws(T, V, topk);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return QUADS_EWORKSPACE;
    const int parts = head::row_parts(T, V, dtype, topk > 0 ? head::kWholeTop : head::kWhole);
    const head::Out o{ids, inv_temp, (int)topk, logp, entropy, stats, top_logp, top_id};
    const head::Parts p{(float4*)ws, (uint64_t*)((char*)ws + 16 * T * parts)};
    if (dtype == QUADS_OUT_BF16)
        head::launch_forward<1>(logits, T, V, ld, parts, o, p, (hipStream_t)stream);
    else
        head::launch_forward<0>(logits, T, V, ld, parts, o, p, (hipStream_t)stream);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

extern "C" int quads_token_logprob_backward(const void* logits, int dtype, int64_t T, int64_t V,
                                            int64_t ld, const int32_t* ids, float inv_temp,
                                            const float* stats, const float* entropy,
                                            const float* g_logp, const float* g_entropy,
                                            void* dlogits, void* stream) {
    const int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!head::ok_opt4(ids) || !ok_ptr4(stats) || !head::ok_opt4(entropy) ||
        !head::ok_opt4(g_logp) || !head::ok_opt4(g_entropy) || !ok_ptr(dlogits))
        return QUADS_EINVAL;
    if ((g_logp != nullptr && ids == nullptr) || (g_entropy != nullptr && entropy == nullptr))
        return QUADS_EINVAL;
    const int parts = head::grad_parts(T, V, dtype);
    const dim3 grid((unsigned)(T * parts)), block(head::kThreads);
    hipStream_t st = (hipStream_t)stream;
    if (dtype == QUADS_OUT_BF16)
        hipLaunchKernelGGL(head::k_logprob_bwd<1>, grid, block, 0, st, logits, V, ld, parts, ids,
                           inv_temp, stats, entropy, g_logp, g_entropy, dlogits);
    else
        hipLaunchKernelGGL(head::k_logprob_bwd<0>, grid, block, 0, st, logits, V, ld, parts, ids,
                           inv_temp, stats, entropy, g_logp, g_entropy, dlogits);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}
