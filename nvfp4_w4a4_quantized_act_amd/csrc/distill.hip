// Distillation from another model's top alternatives and its gradient
// (include/quads_head.h).
//
//   loss = w sum_i q_i (ln q_i - ln p_{id_i}),   dz_v = g w it (Q p_v - q_v)
//
// The list is at most two entries per lane of a wave, so that a wave forms q
// and Q by itself.  The gradient is dense in Q p and differs from it at the
// list's ids alone: those entries are worked out apart, from the logits read
// before anything is written (dlogits may be the logits), and written over
// the dense ones after a barrier.
//
// Loss and gradient in one call go through k_distill_row, which reads each row
// once: see there.  The loss alone and the gradient alone stream a row, or its
// parts where there are few rows (logits.h): k_distill_loss, k_distill_join,
// k_distill_bwd.
#include "logits.h"

namespace quads {
namespace head {

struct List {
    const float* val;
    const int32_t* id;
    const float* weight;
    int topk, renorm;
};

// A lane's two entries of a row's list: q = 0 and ln q = -inf where there is
// none; Q over the wave.
struct Teacher {
    double lq[2];
    float q[2], all;
    int id[2];
};
struct Entries {
    float val[2];
    int id[2];
};
__device__ __forceinline__ Entries load_entries(const List& l, int64_t t) {
    Entries x;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int i = (threadIdx.x & 63) + 64 * b;
        x.id[b] = i < l.topk ? l.id[t * l.topk + i] : -1;
        x.val[b] = i < l.topk ? l.val[t * l.topk + i] : 0.0f;
    }
    return x;
}
// renorm: the list's largest value is subtracted before the product with it,
// in fp64, and the difference rounded once: it * val may be of any size, and
// from 1e9 on its own rounding to fp32 is more than exp spans.  The largest
// entry is then exactly 1 and the sum at least 1.  (One exponential for both
// kinds of list: with one for each, and a second copy of q and ln q, the bf16 row
// kernel of 1024 threads took 481 instead of 458 us at 4096 x 131072.)
__device__ __forceinline__ Teacher teacher(const Entries& x, int V, float it, int renorm) {
    Teacher r;
    float y[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const bool have = x.id[b] >= 0 && x.id[b] < V;
        r.id[b] = have ? x.id[b] : -1;
        y[b] = have ? x.val[b] : -INFINITY;
    }
    const float m = renorm ? stat_base(wave_max(fmaxf(y[0], y[1]))) : 0.0f;
    const double f = renorm ? (double)it : 1.0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        r.lq[b] = f * ((double)y[b] - (double)m);
        r.q[b] = expf((float)r.lq[b]);
    }
    r.all = wave_sum(r.q[0] + r.q[1]);
    if (renorm && r.all != 0.0f) {             // an empty list has nothing to normalise
        const double ls = ln_wide(r.all);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            r.lq[b] -= ls;
            r.q[b] /= r.all;
        }
        r.all = wave_sum(r.q[0] + r.q[1]);
    }
    return r;
}

// The logits at a lane's entries (-inf where there is none).
template <int kBf16>
__device__ __forceinline__ void gather(const Row<kBf16>& r, const Teacher& a, float z[2]) {
#pragma unroll
    for (int b = 0; b < 2; ++b) z[b] = a.id[b] >= 0 ? r.entry(a.id[b]) : -INFINITY;
}

// A row's list, the logits at its ids and their gradients, in LDS while the row
// is worked on (one wave writes and reads it; `all` is for every wave).
struct Parked {
    double lq[QUADS_TOP_MAX];
    int id[QUADS_TOP_MAX];
    float q[QUADS_TOP_MAX], z[QUADS_TOP_MAX], g[QUADS_TOP_MAX];
    float all;
};
__device__ __forceinline__ void park(const Teacher& a, const float z[2], Parked& p) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int i = (threadIdx.x & 63) + 64 * b;
        p.lq[i] = a.lq[b];
        p.id[i] = a.id[b];
        p.q[i] = a.q[b];
        p.z[i] = z[b];
    }
    if ((threadIdx.x & 63) == 0) p.all = a.all;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// sum_i q_i (ln q_i - ln p_i) over the wave.
__device__ __forceinline__ float cross(const Parked& p, float m, double ls, float it) {
    float y = 0.0f;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int i = (threadIdx.x & 63) + 64 * b;
        const float q = p.q[i];
        if (!(q == 0.0f)) y += q * (float)(p.lq[i] - ln_p(p.z[i], m, ls, it));
    }
    return wave_sum(y);
}

// Gradients at the list's ids: by (Q p - q), p = 2^((z - base) cl) inv with inv
// the reciprocal of the row's sum, q summed over the entries with
// the same id in the list's order, so that every one of them has the same
// value.  One wave; they stay in LDS until the dense ones are written.
__device__ __forceinline__ void at_entries(Parked& p, int topk, float by, bool none, float base,
                                           float cl, float inv) {
    const int lane = threadIdx.x & 63;
    const int id[2] = {p.id[lane], p.id[lane + 64]};
    float q[2] = {0.0f, 0.0f};
    for (int i = 0; i < topk; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) q[b] += p.id[i] == id[b] ? p.q[i] : 0.0f;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int i = lane + 64 * b;
        const float x = __builtin_amdgcn_exp2f((p.z[i] - base) * cl) * inv;
        p.g[i] = none ? 0.0f : by * __builtin_fmaf(p.all, x, -q[b]);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}
template <int kBf16>
__device__ __forceinline__ void patch(const Row<kBf16>& r, char* at, const Parked& p, int v0,
                                      int v1) {
    for (int i = threadIdx.x; i < QUADS_TOP_MAX; i += 64) {
        const int v = p.id[i];
        if (v >= v0 && v < v1) {
            if (kBf16)
                ((uint16_t*)at)[r.shift + v] = __builtin_bit_cast(uint16_t, (__bf16)p.g[i]);
            else
                ((float*)at)[r.shift + v] = p.g[i];
        }
    }
}

// One vector's gradient by Q p, a = by Q inv.
template <int kBf16>
__device__ __forceinline__ uint4 dense(const uint4& q, float base, float cl, float a) {
    float g[8];
#pragma unroll
    for (int e = 0; e < Row<kBf16>::kPer; ++e)
        g[e] = a * __builtin_amdgcn_exp2f((get<kBf16>(q, e) - base) * cl);
    return put<kBf16>(g);
}
template <int kBf16>
__device__ __forceinline__ float vec_max(const uint4& q, float m) {
#pragma unroll
    for (int e = 0; e < Row<kBf16>::kPer; ++e) m = fmaxf(m, get<kBf16>(q, e));
    return m;
}
template <int kBf16>
__device__ __forceinline__ float vec_sum(const uint4& q, float base, float cl, float s) {
#pragma unroll
    for (int e = 0; e < Row<kBf16>::kPer; ++e)
        s += __builtin_amdgcn_exp2f((get<kBf16>(q, e) - base) * cl);
    return s;
}

// A vector that the compiler must take as new: without it the fp32 values of
// one pass over a row kept in registers would be kept for the next one too,
// three times the registers.
__device__ __forceinline__ void pin(uint4& q) {
    asm volatile("" : "+v"(q.x), "+v"(q.y), "+v"(q.z), "+v"(q.w));
}

// ------------------------------------------------------------------ streaming --

// Loss and stats of a row from its statistics (one wave).
__device__ __forceinline__ void finish_loss(int64_t t, const Stat& a, const Teacher& q,
                                            const float z[2], float w, float it, float* loss,
                                            float* stats, Parked& p) {
    park(q, z, p);
    const double ls = log_sum(a);
    const float y = cross(p, a.m, ls, it);
    if ((threadIdx.x & 63) == 0) {
        loss[t] = w * y;
        stats[2 * t] = a.m;
        stats[2 * t + 1] = (float)ls;
    }
}
__device__ __forceinline__ void no_loss(int64_t t, float* loss, float* stats) {
    loss[t] = 0.0f;
    stats[2 * t] = 0.0f;
    stats[2 * t + 1] = 0.0f;
}

template <int kBf16, int kThr>
__global__ __launch_bounds__(kThr) void k_distill_loss(const void* z, int64_t V, int64_t ld,
                                                       int parts, List l, float it, float* loss,
                                                       float* stats, float4* part_stat) {
    constexpr int kChunk = kThr * kVecs;
    __shared__ Stat s_stat[kThr / 64];
    __shared__ Parked s_list;
    const int64_t t = blockIdx.x / (unsigned)parts;
    const int part = (int)(blockIdx.x % (unsigned)parts);
    const float w = l.weight ? l.weight[t] : 1.0f;
    if (w == 0.0f) {
        if (parts == 1 && threadIdx.x == 0) no_loss(t, loss, stats);
        return;
    }
    const Row<kBf16> r(z, t, ld, V);
    const float cl = it * kLog2e;
    const int chunks = (r.nvec + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * part / parts);
    const int c1 = (int)((int64_t)chunks * (part + 1) / parts);
    auto load = [&](uint4 (&q)[kVecs], int ch) {
        if (ch >= c1) return;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = ch * kChunk + i * kThr + threadIdx.x;
            if (r.whole(j)) q[i] = *r.vec(j);
            else q[i] = r.part(j);
        }
    };
    Stat a = {-INFINITY, 0.0f, 0.0f};
    uint4 q[kVecs], next[kVecs];
    // the list and the logits at its ids come while the row is read
    const bool first = parts == 1 && threadIdx.x < 64;
    Entries x = {};
    if (first) x = load_entries(l, t);
    load(next, c0);
    Teacher list = {};
    float zq[2] = {0.0f, 0.0f};
    if (first) {
        list = teacher(x, r.V, it, l.renorm);
        gather<kBf16>(r, list, zq);
    }
    for (int ch = c0; ch < c1; ++ch) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) q[i] = next[i];
        load(next, ch + 1);
        float m = a.m;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) m = vec_max<kBf16>(q[i], m);
        stat_raise(a, m, cl);
        const float base = stat_base(m);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) a.s = vec_sum<kBf16>(q[i], base, cl, a.s);
    }
    a = group_stat<kThr / 64>(a, cl, s_stat);
    if (parts > 1) {
        if (threadIdx.x == 0) part_stat[blockIdx.x] = make_float4(a.m, a.s, 0.0f, 0.0f);
    } else if (first) {
        finish_loss(t, a, list, zq, w, it, loss, stats, s_list);
    }
}

// Joins the parts of a row: one wave, lane l part l.
template <int kBf16>
__global__ __launch_bounds__(64) void k_distill_join(const void* z, int64_t V, int64_t ld,
                                                     int parts, List l, float it, float* loss,
                                                     float* stats, const float4* part_stat) {
    __shared__ Parked s_list;
    const int64_t t = blockIdx.x;
    const float w = l.weight ? l.weight[t] : 1.0f;
    if (w == 0.0f) {
        if (threadIdx.x == 0) no_loss(t, loss, stats);
        return;
    }
    const Row<kBf16> r(z, t, ld, V);
    const Entries x = load_entries(l, t);
    Stat a = {-INFINITY, 0.0f, 0.0f};
    if ((int)threadIdx.x < parts) {
        const float4 q = part_stat[t * parts + threadIdx.x];
        a = {q.x, q.y, q.z};
    }
    const Teacher list = teacher(x, r.V, it, l.renorm);
    float zq[2];
    gather<kBf16>(r, list, zq);
    a = wave_stat(a, it * kLog2e);
    finish_loss(t, a, list, zq, w, it, loss, stats, s_list);
}

template <int kBf16, int kThr>
__global__ __launch_bounds__(kThr) void k_distill_bwd(const void* z, int64_t V, int64_t ld,
                                                      int parts, List l, float it,
                                                      const float* stats, const float* g,
                                                      void* dz) {
    constexpr int kChunk = kThr * kVecs;
    __shared__ Parked s_list;
    const int64_t t = blockIdx.x / (unsigned)parts;
    const int part = (int)(blockIdx.x % (unsigned)parts);
    const Row<kBf16> r(z, t, ld, V);
    char* out = (char*)dz + (r.at - (const char*)z);
    const int chunks = (r.nvec + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * part / parts);
    const int c1 = (int)((int64_t)chunks * (part + 1) / parts);
    const float w = l.weight ? l.weight[t] : 1.0f;
    if (w == 0.0f) {
        for (int j = c0 * kChunk + threadIdx.x; j < c1 * kChunk && j < r.nvec; j += kThr)
            store_vec<kBf16>(r, out, j, make_uint4(0, 0, 0, 0));
        return;
    }
    // the first chunk comes while the list is worked on
    uint4 x[kVecs];
    auto load = [&](int ch) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = ch * kChunk + i * kThr + threadIdx.x;
            if (r.whole(j)) x[i] = *r.vec(j);
            else x[i] = r.part(j);
        }
    };
    const Entries listed = load_entries(l, t);
    const float m = stats[2 * t], ls = stats[2 * t + 1];
    const float by = w * it * (g ? g[t] : 1.0f);
    load(c0);
    const Teacher q = teacher(listed, r.V, it, l.renorm);
    const float base = stat_base(m), cl = it * kLog2e, inv = recip_sum(ls);
    // the part's entries [v0, v1), their gradients parked before any store.  In
    // place, a logit that lies in another part may already be its gradient: what
    // is worked out from it is not used (patch), and nothing else reads it.
    const int v0 = c0 ? r.index(c0 * kChunk, 0) : 0, v1 = r.index(c1 * kChunk, 0);
    if (threadIdx.x < 64) {
        float zq[2];
        gather<kBf16>(r, q, zq);
        park(q, zq, s_list);
        at_entries(s_list, l.topk, by, m == -INFINITY && ls == ls, base, cl, inv);
    }
    __syncthreads();
    const float a = by * q.all * inv;
    for (int ch = c0; ch < c1; ++ch) {
        if (ch > c0) load(ch);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int j = ch * kChunk + i * kThr + threadIdx.x;
            if (j < r.nvec) store_vec<kBf16>(r, out, j, dense<kBf16>(x[i], base, cl, a));
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) patch<kBf16>(r, out, s_list, v0, v1);
}

// ------------------------------------------------------- loss and gradient --

__device__ __forceinline__ void st_stream16(char* p, const uint4& q) {
    __builtin_nontemporal_store((u32x4){q.x, q.y, q.z, q.w}, reinterpret_cast<u32x4*>(p));
}

// One row at a time, read once: a thread keeps kNv of the row's vectors in
// registers between the log-sum and the gradient (a CU's registers hold 256
// KB of a row: 131072 bf16 or 65536 fp32 entries); what a longer row has
// beyond them is read a second time.  The work-groups are resident ones that
// walk over the rows: a vector of the next row is requested into the registers
// of the one whose gradient was just stored, so that loads, stores and
// arithmetic overlap although a CU holds one row at a time.  The partial
// vectors at a row's ends are in one more register vector of threads 0 and 1.
// With 1024 threads the compiler spills up to 5 of 128 registers (24 bytes of
// scratch a lane): stored before the loop over the rows, read back once or twice
// per row in the joins and the list's work, not in the passes over the vectors.
//
// kLong (rows beyond the registers): what is read or written once is marked
// as not to be kept, so that the cache keeps the part that is read again (1000
// x 100001 fp32: 189 -> 173 us, 512 x 100000: 95 -> 81, 1000 x 200000 bf16: 194
// -> 192; shorter rows gain or lose by it, from 111 -> 121 us at 4096 x 30000
// bf16 to 394 -> 379 at 4096 x 60000 fp32, and do without).
template <int kBf16, int kThr, int kNv, bool kLong>
__global__ __launch_bounds__(kThr, 4) void k_distill_row(const void* z, int64_t T, int64_t V,
                                                      int64_t ld, List l, float it, float* loss,
                                                      void* dz) {
    constexpr int kPer = Row<kBf16>::kPer;
    __shared__ Stat s_stat[kThr / 64];
    __shared__ Parked s_list;
    const uint4 masked = kBf16 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                               : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    const float cl = it * kLog2e;
    const int tid = threadIdx.x;

    uint4 x[kNv], edge;
    // the whole vectors of a row are first .. first + count - 1
    auto first = [](const Row<kBf16>& r) { return r.shift ? 1 : 0; };
    auto count = [](const Row<kBf16>& r) { return (r.V + r.shift) / kPer - (r.shift ? 1 : 0); };
    // the partial vector this thread holds, or -1
    auto edge_at = [&](const Row<kBf16>& r) {
        const int last = (r.V + r.shift) % kPer ? r.nvec - 1 : -1;
        if (tid == 0) return r.shift ? 0 : -1;
        return tid == 1 && (last > 0 || !r.shift) ? last : -1;
    };
    // vector i of the `n` whole ones of a row, -inf past them; addressed as a
    // uniform base plus 16 tid (one register)
    const uint32_t lane16 = 16u * (uint32_t)tid;
    auto load = [&](const Row<kBf16>& r, int n, int i) {
        const char* at = r.at + 16 * (int64_t)(first(r) + i * kThr);
        x[i] = masked;
        if (i * kThr + tid < n)
            x[i] = kLong ? ld_stream16(at + lane16) : *reinterpret_cast<const uint4*>(at + lane16);
    };
    auto load_edge = [&](const Row<kBf16>& r, bool live) {
        const int j = live ? edge_at(r) : -1;
        edge = masked;
        if (j >= 0) edge = r.part(j);
    };

    int64_t t = blockIdx.x;
    Entries e = load_entries(l, t);
    float w = l.weight ? l.weight[t] : 1.0f;
    {
        const Row<kBf16> r(z, t, ld, V);
        load_edge(r, w != 0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) load(r, w != 0.0f ? count(r) : 0, i);
    }
    for (; t < T; t += gridDim.x) {
        const Row<kBf16> r(z, t, ld, V);
        char* out = (char*)dz + (r.at - (const char*)z);
        // the next row's list and weight; a row of weight 0 is not read but
        // taken as masked throughout, which gives the gradient 0
        const int64_t tn = t + gridDim.x < T ? t + gridDim.x : t;
        const Entries en = load_entries(l, tn);
        const float wn = l.weight ? l.weight[tn] : 1.0f;
        const Row<kBf16> rn(z, tn, ld, V);
        const bool more = tn != t && wn != 0.0f;
        const int n = count(r), beyond = w != 0.0f ? n : 0, nn = more ? count(rn) : 0;

        if (tid < 64) {
            Teacher q = teacher(e, r.V, it, l.renorm);
            if (w == 0.0f) q.id[0] = q.id[1] = -1;
            float zq[2];
            gather<kBf16>(r, q, zq);
            park(q, zq, s_list);
        }
        // log-sum: the vectors in registers, then those beyond them
        Stat a = {vec_max<kBf16>(edge, -INFINITY), 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kNv; ++i)
            if (i * kThr < n) {
                a.m = vec_max<kBf16>(x[i], a.m);
                pin(x[i]);
            }
        float base = stat_base(a.m);
        a.s = vec_sum<kBf16>(edge, base, cl, 0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i)
            if (i * kThr < n) {
                a.s = vec_sum<kBf16>(x[i], base, cl, a.s);
                pin(x[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        for (int i = kNv * kThr + tid; kLong && i < beyond; i += kThr) {
            const uint4 y = *r.vec(first(r) + i);
            stat_raise(a, vec_max<kBf16>(y, a.m), cl);
            a.s = vec_sum<kBf16>(y, stat_base(a.m), cl, a.s);
        }
        a = group_stat<kThr / 64>(a, cl, s_stat);
        const bool none = a.m == -INFINITY && a.s == 0.0f;
        base = stat_base(a.m);
        const float by = w * it, inv = none ? 0.0f : 1.0f / a.s;
        if (tid < 64) {
            const float y = cross(s_list, a.m, log_sum(a), it);
            if (tid == 0) loss[t] = w == 0.0f ? 0.0f : w * y;
            at_entries(s_list, l.topk, by, none, base, cl, inv);
        }
        // gradient
        const float f = w == 0.0f ? 0.0f : by * s_list.all * inv;
        for (int i = kNv * kThr + tid; kLong && i < n; i += kThr) {
            const int j = first(r) + i;
            uint4 y = masked;
            if (i < beyond) y = *r.vec(j);
            st_stream16(out + 16 * (int64_t)j, dense<kBf16>(y, base, cl, f));
        }
        const int j = edge_at(r);
        if (j >= 0) store_part<kBf16>(r, out, j, dense<kBf16>(edge, base, cl, f));
        load_edge(rn, more);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (i * kThr < n) {
                const uint4 y = dense<kBf16>(x[i], base, cl, f);
                char* to = out + 16 * (int64_t)(first(r) + i * kThr);
                if (i * kThr + tid < n) {
                    if (kLong) st_stream16(to + lane16, y);
                    else *reinterpret_cast<uint4*>(to + lane16) = y;
                }
            }
            load(rn, nn, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
        if (tid < 64) patch<kBf16>(r, out, s_list, 0, r.V);
        e = en;
        w = wn;
    }
}

inline int check_list(int64_t T, const float* t_val, const int32_t* t_id, int32_t topk,
                      const float* weight, int renorm) {
    if (topk < 1 || topk > QUADS_TOP_MAX) return QUADS_ESHAPE;
    if (renorm != 0 && renorm != 1) return QUADS_EINVAL;
    if (T == 0) return QUADS_OK;
    return ok_ptr4(t_val) && ok_ptr4(t_id) && ok_opt4(weight) ? QUADS_OK : QUADS_EINVAL;
}

// The work-group of k_distill_row: the smallest whose registers hold a row of
// nvec vectors (4096 x 2000 bf16: 16 us with 64 threads, 21 with 128, 33 with
// 256), and how many of them are resident together.
constexpr int kCus = 256;
constexpr int kRowVecs = 16;                   // vectors of a row per thread
inline int row_threads(int64_t nvec) {
    int n = 64;
    while (n < 1024 && nvec > kRowVecs * n) n *= 2;
    return n;
}
inline int64_t row_slots(int64_t nvec) { return (int64_t)kCus * (1024 / row_threads(nvec)); }
// Whether loss and gradient take k_distill_row: always, but for a few rows that
// are longer than a work-group's registers, which are split.  In us, row by row
// / split: 1 x 20000 bf16 13 / 20, 64 x 100001 fp32 23 / 25, 64 x 140001 30 / 37,
// 300 x 140001 99 / 119, 600 x 300001 410 / 485; bf16 64 x 140001 30 / 26, 300 x
// 140001 70 / 68, 600 x 140001 109 / 119.  A row by row form with fewer rows than
// CUs leaves CUs without one, and reads what is beyond the registers twice: from
// about 300000 entries on the split would be the better one (fp32 64 x 300001 86
// / 62, 64 x 1000003 300 / 183, 300 x 1000003 894 / 802; bf16 128 x 1000003 207 /
// 170), which the rule, made for vocabularies up to 131072, does not see.
inline bool whole_rows(int64_t T, int64_t V, int dtype) {
    return T >= 64 || row_vectors(V, dtype) <= kRowVecs * 1024;
}

// Vectors of a row that a wave takes alone (short_rows; in us, calls in turn
// from a graph, 256 / 64 threads; loss: 4096 x 1227 fp32 14.0 / 10.3, 4096 x 4000
// 17.9 / 16.5, 4096 x 2000 bf16 17.7 / 9.2, not for 1024 x 4000 fp32 7.1 / 7.5;
// gradient: 4096 x 300 fp32 16.5 / 9.6, 4096 x 2000 bf16 20.9 / 15.4, not for
// 4096 x 2000 fp32 22.7 / 25.6).
constexpr int kShortLoss = 1024, kShortGrad = 256;

template <int kBf16>
void launch_loss(const void* z, int64_t T, int64_t V, int64_t ld, const List& l, float it,
                 float* loss, float* stats, void* ws, hipStream_t st) {
    const int parts = row_parts(T, V, kBf16 ? QUADS_OUT_BF16 : QUADS_OUT_F32, kWhole);
    if (short_rows(T, row_vectors(V, kBf16 ? QUADS_OUT_BF16 : QUADS_OUT_F32), kShortLoss))
        hipLaunchKernelGGL((k_distill_loss<kBf16, 64>), dim3((unsigned)T), dim3(64), 0, st, z, V,
                           ld, 1, l, it, loss, stats, (float4*)nullptr);
    else if (wide_rows<kBf16>(T, V, parts))
        hipLaunchKernelGGL((k_distill_loss<kBf16, kWideThreads>), dim3((unsigned)T),
                           dim3(kWideThreads), 0, st, z, V, ld, 1, l, it, loss, stats, (float4*)nullptr);
    else
        hipLaunchKernelGGL((k_distill_loss<kBf16, kThreads>), dim3((unsigned)(T * parts)),
                           dim3(kThreads), 0, st, z, V, ld, parts, l, it, loss, stats,
                           (float4*)ws);
    if (parts > 1)
        hipLaunchKernelGGL(k_distill_join<kBf16>, dim3((unsigned)T), dim3(64), 0, st, z, V, ld,
                           parts, l, it, loss, stats, (const float4*)ws);
}
template <int kBf16>
void launch_bwd(const void* z, int64_t T, int64_t V, int64_t ld, const List& l, float it,
                const float* stats, const float* g, void* dz, hipStream_t st) {
    const int parts = grad_parts(T, V, kBf16 ? QUADS_OUT_BF16 : QUADS_OUT_F32);
    if (short_rows(T, row_vectors(V, kBf16 ? QUADS_OUT_BF16 : QUADS_OUT_F32), kShortGrad))
        hipLaunchKernelGGL((k_distill_bwd<kBf16, 64>), dim3((unsigned)T), dim3(64), 0, st, z, V, ld,
                           1, l, it, stats, g, dz);
    else
        hipLaunchKernelGGL((k_distill_bwd<kBf16, kThreads>), dim3((unsigned)(T * parts)),
                           dim3(kThreads), 0, st, z, V, ld, parts, l, it, stats, g, dz);
}
template <int kBf16>
void launch_row(const void* z, int64_t T, int64_t V, int64_t ld, const List& l, float it,
                float* loss, void* dz, hipStream_t st) {
    const int64_t nvec = row_vectors(V, kBf16 ? QUADS_OUT_BF16 : QUADS_OUT_F32);
    const int thr = row_threads(nvec);
    const int64_t slots = row_slots(nvec);
    const dim3 grid((unsigned)(T < slots ? T : slots)), block(thr);
#define QUADS_ROW(THR, LONG)                                                                  \
    hipLaunchKernelGGL((k_distill_row<kBf16, THR, kRowVecs, LONG>), grid, block, 0, st, z, T, V, \
                       ld, l, it, loss, dz)
    if (thr == 64) QUADS_ROW(64, false);
    else if (thr == 128) QUADS_ROW(128, false);
    else if (thr == 256) QUADS_ROW(256, false);
    else if (thr == 512) QUADS_ROW(512, false);
    else if (nvec <= kRowVecs * 1024) QUADS_ROW(1024, false);
    else QUADS_ROW(1024, true);
#undef QUADS_ROW
}

// The parts' statistics.
inline size_t parts_ws(int64_t T, int64_t V) {
    const int parts = row_parts(T, V, QUADS_OUT_F32, kWhole);
    return parts > 1 ? (size_t)T * parts * 16 : 0;
}

}  // namespace head
}  // namespace quads

using namespace quads;

extern "C" size_t quads_topk_distill_ws(int64_t T, int64_t V, int32_t topk) {
    return T < 1 || V < 1 || topk < 1 ? 0 : head::parts_ws(T, V);
}

// The split rows' statistics, then the stats their second step reads (whether
// rows are split depends on the type: as much as either needs).
extern "C" size_t quads_topk_distill_grad_ws(int64_t T, int64_t V, int32_t topk) {
    if (T < 1 || V < 1 || topk < 1 || head::whole_rows(T, V, QUADS_OUT_F32)) return 0;
    return head::parts_ws(T, V) + (size_t)T * 8;
}

extern "C" int quads_topk_distill(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                  const float* t_val, const int32_t* t_id, int32_t topk,
                                  const float* weight, float inv_temp, int renorm, float* loss,
                                  float* stats, void* ws, size_t ws_bytes, void* stream) {
    int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc == QUADS_OK) rc = head::check_list(T, t_val, t_id, topk, weight, renorm);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!ok_ptr4(loss) || !ok_ptr4(stats)) return QUADS_EINVAL;
    const size_t need = quads_topk_distill_ws(T, V, topk);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return QUADS_EWORKSPACE;
    const head::List l{t_val, t_id, weight, (int)topk, renorm};
    if (dtype == QUADS_OUT_BF16)
        head::launch_loss<1>(logits, T, V, ld, l, inv_temp, loss, stats, ws, (hipStream_t)stream);
    else
        head::launch_loss<0>(logits, T, V, ld, l, inv_temp, loss, stats, ws, (hipStream_t)stream);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

extern "C" int quads_topk_distill_backward(const void* logits, int dtype, int64_t T, int64_t V,
                                           int64_t ld, const float* t_val, const int32_t* t_id,
                                           int32_t topk, const float* weight, float inv_temp,
                                           int renorm, const float* stats, const float* g,
                                           void* dlogits, void* stream) {
    int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc == QUADS_OK) rc = head::check_list(T, t_val, t_id, topk, weight, renorm);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!ok_ptr4(stats) || !ok_ptr4(g) || !ok_ptr(dlogits)) return QUADS_EINVAL;
    const head::List l{t_val, t_id, weight, (int)topk, renorm};
    if (dtype == QUADS_OUT_BF16)
        head::launch_bwd<1>(logits, T, V, ld, l, inv_temp, stats, g, dlogits, (hipStream_t)stream);
    else
        head::launch_bwd<0>(logits, T, V, ld, l, inv_temp, stats, g, dlogits, (hipStream_t)stream);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

extern "C" int quads_topk_distill_grad(const void* logits, int dtype, int64_t T, int64_t V,
                                       int64_t ld, const float* t_val, const int32_t* t_id,
                                       int32_t topk, const float* weight, float inv_temp,
                                       int renorm, float* loss, void* dlogits, void* ws,
                                       size_t ws_bytes, void* stream) {
    int rc = head::check_rows(logits, dtype, T, V, ld, inv_temp);
    if (rc == QUADS_OK) rc = head::check_list(T, t_val, t_id, topk, weight, renorm);
    if (rc != QUADS_OK || T == 0) return rc;
    if (!ok_ptr4(loss) || !ok_ptr(dlogits)) return QUADS_EINVAL;
    const size_t need = quads_topk_distill_grad_ws(T, V, topk);
    if (ws_bytes < need || (need > 0 && !ok_ptr(ws))) return QUADS_EWORKSPACE;
    const head::List l{t_val, t_id, weight, (int)topk, renorm};
    hipStream_t st = (hipStream_t)stream;
    const bool bf16 = dtype == QUADS_OUT_BF16;
    if (head::whole_rows(T, V, dtype)) {
        if (bf16) head::launch_row<1>(logits, T, V, ld, l, inv_temp, loss, dlogits, st);
        else head::launch_row<0>(logits, T, V, ld, l, inv_temp, loss, dlogits, st);
    } else {
        float* stats = (float*)((char*)ws + head::parts_ws(T, V));
        if (bf16) {
            head::launch_loss<1>(logits, T, V, ld, l, inv_temp, loss, stats, ws, st);
            head::launch_bwd<1>(logits, T, V, ld, l, inv_temp, stats, nullptr, dlogits, st);
        } else {
            head::launch_loss<0>(logits, T, V, ld, l, inv_temp, loss, stats, ws, st);
            head::launch_bwd<0>(logits, T, V, ld, l, inv_temp, stats, nullptr, dlogits, st);
        }
    }
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}
