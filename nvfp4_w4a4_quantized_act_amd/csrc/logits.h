// Pieces shared by the kernels that read the output head's logits
// (include/quads_head.h): rows of any alignment in 16-byte vectors, the
// running softmax statistics, and the host-side checks.
#pragma once

#include "common.h"
#include "../../include/quads_head.h"

namespace quads {
namespace head {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
// A term 2^d with d below this is 0 in fp32; d is clamped here where it is a
// factor (0 * -inf would be NaN).
constexpr float kNoTerm = -200.0f;

// Logits [T, V] with row stride ld.  A row is read in 16-byte vectors at
// 16-byte boundaries: vector j holds the entries j * kPer - shift + (0 ..
// kPer - 1), shift the entries between the boundary before the row and its
// first one.  The first and the last vector may be partial.
template <int kBf16>
struct Row {
    static constexpr int kPer = kBf16 ? 8 : 4;
    const char* at;                       // the boundary at or before the row
    int shift, V, nvec;

    __device__ __forceinline__ Row(const void* z, int64_t t, int64_t ld, int64_t v) {
        const int64_t first = t * ld;
        shift = (int)(first & (kPer - 1));
        at = (const char*)z + (first - shift) * (16 / kPer);
        V = (int)v;
        nvec = (int)((v + shift + kPer - 1) / kPer);
    }
    __device__ __forceinline__ int index(int j, int i) const { return j * kPer + i - shift; }
    __device__ __forceinline__ bool whole(int j) const {
        return index(j, 0) >= 0 && index(j, kPer - 1) < V;
    }
    // vector j of the row; entries outside the row read as -inf
    __device__ __forceinline__ uint4 part(int j) const {
        uint4 r = kBf16 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                        : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
        uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = index(j, i);
            if (v >= 0 && v < V) {
                if (kBf16) {
                    const uint32_t h = ((const uint16_t*)at)[(int64_t)j * kPer + i];
                    w[i >> 1] = (i & 1) ? (w[i >> 1] & 0xFFFFu) | (h << 16)
                                        : (w[i >> 1] & 0xFFFF0000u) | h;
                } else {
                    w[i] = ((const uint32_t*)at)[(int64_t)j * kPer + i];
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ const uint4* vec(int j) const {
        return reinterpret_cast<const uint4*>(at) + j;
    }
    __device__ __forceinline__ float entry(int64_t v) const {
        return kBf16 ? bf16_to_f32(((const uint16_t*)at)[shift + v])
                     : ((const float*)at)[shift + v];
    }
};

// Entry i of a vector in fp32.
template <int kBf16>
__device__ __forceinline__ float get(const uint4& q, int i) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if (kBf16) return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    return __uint_as_float(w[i]);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
template <int kBf16>
__device__ __forceinline__ uint4 put(const float* g) {
    if (kBf16)
        return make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]),
                          pack_bf16(g[6], g[7]));
    return make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                      __float_as_uint(g[3]));
}
// Stores the entries of vector j that lie in the row (`at` as Row::at, of the output).
template <int kBf16>
__device__ __forceinline__ void store_part(const Row<kBf16>& r, char* at, int j, const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < Row<kBf16>::kPer; ++i) {
        const int v = r.index(j, i);
        if (v >= 0 && v < r.V) {
            if (kBf16)
                ((uint16_t*)at)[(int64_t)j * 8 + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            else
                ((uint32_t*)at)[(int64_t)j * 4 + i] = w[i];
        }
    }
}
template <int kBf16>
__device__ __forceinline__ void store_vec(const Row<kBf16>& r, char* at, int j, const uint4& q) {
    if (r.whole(j)) reinterpret_cast<uint4*>(at)[j] = q;
    else store_part<kBf16>(r, at, j, q);
}

// Running statistics of some entries: m = max z, and with d = c (z - m),
// c = it log2(e):  s = sum 2^d, u = sum 2^d d.  Rescaled when m rises, one
// pass over the data.  Entries of -inf add nothing; m = -inf, s = 0 while
// there is no other.  c is one fp32 number, up to 7e-8 off: every d is off by
// that share of itself and ln s by at most that times sum p |d| (1e-8 of it at
// it = 1, 3e-8 at 1.3).  The rest of c would be one more operation per entry of
// kernels whose vector units are up to 89% busy.
struct Stat {
    float m, s, u;
};
__device__ __forceinline__ float stat_base(float m) { return m == -INFINITY ? 0.0f : m; }

// `a` with its maximum raised to m (m >= a.m).
__device__ __forceinline__ void stat_raise(Stat& a, float m, float c) {
    const float d = __builtin_amdgcn_fmed3f((stat_base(a.m) - stat_base(m)) * c, kNoTerm, 0.0f);
    const float r = __builtin_amdgcn_exp2f(d);
    a.u = r * __builtin_fmaf(d, a.s, a.u);
    a.s *= r;
    a.m = m;
}

// Sum and maximum over the 64 lanes of a wave (every lane active), the same bits
// in every lane: DPP moves within the rows of 16 lanes and across them, then
// one lane's value read as a scalar (lane shuffles, through LDS, took ten
// times as long: a row of a loss has ten such reductions one after another).
template <int kCtrl, int kRowMask>
__device__ __forceinline__ float dpp_move(float old, float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        (int)__float_as_uint(old), (int)__float_as_uint(v), kCtrl, kRowMask, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_move<0x111, 0xF>(0.0f, v);        // row_shr:1
    v += dpp_move<0x112, 0xF>(0.0f, v);        // row_shr:2
    v += dpp_move<0x114, 0xF>(0.0f, v);        // row_shr:4
    v += dpp_move<0x118, 0xF>(0.0f, v);        // row_shr:8
    v += dpp_move<0x142, 0xA>(0.0f, v);        // row_bcast:15 into rows 1 and 3
    v += dpp_move<0x143, 0xC>(0.0f, v);        // row_bcast:31 into rows 2 and 3
    return last_lane(v);
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp_move<0x111, 0xF>(v, v));
    v = fmaxf(v, dpp_move<0x112, 0xF>(v, v));
    v = fmaxf(v, dpp_move<0x114, 0xF>(v, v));
    v = fmaxf(v, dpp_move<0x118, 0xF>(v, v));
    v = fmaxf(v, dpp_move<0x142, 0xA>(v, v));
    v = fmaxf(v, dpp_move<0x143, 0xC>(v, v));
    return last_lane(v);
}
__device__ __forceinline__ Stat wave_stat(Stat a, float c) {
    stat_raise(a, wave_max(a.m), c);
    a.s = wave_sum(a.s);
    a.u = wave_sum(a.u);
    return a;
}
// Statistics of the whole work-group, in every thread (s_stat: one per wave).
template <int kWaves>
__device__ __forceinline__ Stat group_stat(Stat a, float c, Stat* s_stat) {
    a = wave_stat(a, c);
    if ((threadIdx.x & 63) == 0) s_stat[threadIdx.x >> 6] = a;
    __syncthreads();
    const int l = threadIdx.x & 63;
    Stat b = {-INFINITY, 0.0f, 0.0f};
    if (l < kWaves) b = s_stat[l];
    return wave_stat(b, c);
}

// ln s to about 2^-24, however large it is: the exponent and the fp32 logarithm
// of the mantissa, added in fp64 (an fp32 logarithm of 2^15 is off by four bits
// of that, and fp64's own takes 30 registers that the kernels do not have).
__device__ __forceinline__ double ln_wide(float s) {
    const double e = (double)__builtin_amdgcn_frexp_expf(s);
    return 0.69314718055994531 * (e + (double)__builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(s)));
}
// ln sum exp(it (z - m)): 0 for a row without an unmasked entry.  In fp64, as is
// what is taken from it, once or a few times per row: a log-probability or a
// small loss is a difference of such numbers.
__device__ __forceinline__ double log_sum(const Stat& a) {
    return a.m == -INFINITY && a.s == 0.0f ? 0.0 : ln_wide(a.s);
}
// 1 / sum exp(it (z - m)) from the fp32 log-sum a forward pass has left, with
// no more error than ls has itself: ls log2(e) in two parts.  A probability is
// then 2^((z - m) cl) times it, which for a large one is nearer than the power
// of the difference.
__device__ __forceinline__ float recip_sum(float ls) {
    const float hi = ls * kLog2e;
    const float lo = __builtin_fmaf(ls, kLog2e, -hi) + ls * 1.92596299e-8f;
    return __builtin_amdgcn_exp2f(-hi) * __builtin_fmaf(-lo, kLn2, 1.0f);
}
// ln p of an entry: -inf where it is masked (unless the row holds NaN or +inf).
__device__ __forceinline__ double ln_p(float z, float m, double ls, float it) {
    return z == -INFINITY && ls == ls ? (double)z : ((double)z - (double)m) * (double)it - ls;
}

// ------------------------------------------------------------------ host --

// Row parts: a row is split over work-groups of kThreads threads where there
// are too few rows to fill the GPU, into parts of whole chunks (kChunk
// vectors).
constexpr int kThreads = 256;
constexpr int kVecs = 4;                       // vectors per thread and chunk
constexpr int kChunk = kThreads * kVecs;
constexpr int kMaxParts = 64;
constexpr int kGroups = 1024;                  // work-groups wanted: four per CU

inline int split_row(int64_t T, int64_t V, int dtype, int64_t groups) {
    const int per = dtype == QUADS_OUT_BF16 ? 8 : 4;
    const int64_t chunks = (V + per - 1 + (int64_t)per * kChunk) / ((int64_t)per * kChunk);
    int64_t p = groups / T;
    if (p > chunks) p = chunks;
    return p < 1 ? 1 : (int)p;
}
// Parts of a row for sums, which a second kernel joins: not for rows of up to
// `whole` entries, whose work-group is done before the host has made a second
// launch.  In us with one work-group a row (wide_rows) / split, calls in turn,
// and in brackets device time from a graph, fp32: no alternatives 1 x 65536
// 11.6 / 16.5 (7.9 / 4.7), 64 x 65536 11.9 / 16.8 (8.7 / 8.3), 1 x 131072 12.5 /
// 16.7 (12.4 / 4.8), 64 x 131072 15.0 / 16.8 (15.0 / 11.2); top 20, 1 x 32768
// 15.0 / 20.0 (10.6 / 9.9), 1 x 50001 17.7 / 19.5 (17.1 / 10.3), 64 x 65536 18.2
// / 19.9 (17.9 / 15.3), 64 x 131072 26.8 / 21.0 (26.6 / 20.6).  From a graph
// fewer rows than about 64 gain by a split from 32768 entries on, and 256 rows
// lose by it at any length (65536 with top 20 22 / 26, 131072 without 27 / 30):
// the rule looks at neither.
constexpr int kWhole = 65536, kWholeTop = 32768;
inline int row_parts(int64_t T, int64_t V, int dtype, int whole) {
    if (V <= whole) return 1;
    const int p = split_row(T, V, dtype, kGroups);
    return p < kMaxParts ? p : kMaxParts;
}
// Rows of one work-group each, at most one per CU and longer than two chunks,
// take a work-group of four times the threads for their sums (in us, calls in
// turn from a graph, 256 / 1024 threads: the distillation's loss 33 x 50001 fp32
// 12.2 / 8.9, 256 x 65536 22.4 / 16.0, 1 x 16000 5.4 / 4.5, 256 x 32000 bf16 7.7
// / 7.2, not for 512 x 50001 bf16 15.5 / 17.7, 33 x 8000 4.6 / 6.2; with the top
// 20 alternatives 128 x 16000 fp32 12.4 / 10.1, 1 x 20000 bf16 11.3 / 10.1).
constexpr int kWideThreads = 1024;
template <int kBf16>
inline bool wide_rows(int64_t T, int64_t V, int parts) {
    return parts == 1 && T <= 256 && V > 2 * kChunk * (int64_t)Row<kBf16>::kPer;
}
// Many short rows take a wave each: what is done once per row is most of the
// work, and three of four waves would wait for it.
inline int64_t row_vectors(int64_t V, int dtype) {
    const int per = dtype == QUADS_OUT_BF16 ? 8 : 4;
    return (V + per - 1) / per;
}
inline bool short_rows(int64_t T, int64_t nvec, int most) { return T >= 2048 && nvec <= most; }
// Parts of a row for a gradient: nothing is joined, so that more of them are
// better, up to what the GPU holds at once (1023 x 50001 fp32, both passes: 145
// us with 1024 work-groups wanted, 141 with 2048, 137 with 4096, 150 with 8192).
inline int grad_parts(int64_t T, int64_t V, int dtype) {
    return split_row(T, V, dtype, 4 * kGroups);
}

inline bool ok_opt4(const void* p) { return p == nullptr || ok_ptr4(p); }

inline int check_rows(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, float it) {
    if (T < 0 || T >= ((int64_t)1 << 24) || V < 1 || V >= ((int64_t)1 << 30) || ld < V ||
        ld >= ((int64_t)1 << 31))
        return QUADS_ESHAPE;
    if (dtype != QUADS_OUT_F32 && dtype != QUADS_OUT_BF16) return QUADS_EINVAL;
    if (!(it > 0.0f) || !(it <= 1e30f)) return QUADS_EINVAL;
    if (T == 0) return QUADS_OK;
    return ok_ptr(logits) ? QUADS_OK : QUADS_EINVAL;
}

}  // namespace head
}  // namespace quads
