// Shared by the kernels of the layer around the experts (quads_block.h): rows
// of channels in bf16 or fp32, read and written eight channels at a time.
//
// A row may start at any element (odd lengths, row strides of the caller's):
// the eight channels of a thread are one 16-byte access (bf16) or two (fp32)
// at whatever address they have, which gfx950 takes (at whole words without a
// loss, at odd bf16 elements 8192 x 5001 84 us against 69).
#pragma once

#include "common.h"
#include "../../include/quads_block.h"

namespace quads {
namespace block {

constexpr int kPer = 8;                      // channels per access

typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef words4 words4_at2 __attribute__((aligned(2), may_alias));
typedef words4 words4_at4 __attribute__((aligned(4), may_alias));
typedef uint32_t words2 __attribute__((ext_vector_type(2)));

// 16 bytes at any element's address.
template <bool kOnce>
__device__ __forceinline__ words4 read(const uint16_t* p) {
    const words4_at2* q = reinterpret_cast<const words4_at2*>(p);
    if (kOnce) return __builtin_nontemporal_load(q);
    return *q;
}
template <bool kOnce>
__device__ __forceinline__ words4 read(const uint32_t* p) {
    const words4_at4* q = reinterpret_cast<const words4_at4*>(p);
    if (kOnce) return __builtin_nontemporal_load(q);
    return *q;
}
template <bool kOnce>
__device__ __forceinline__ void write(uint16_t* p, words4 v) {
    words4_at2* q = reinterpret_cast<words4_at2*>(p);
    if (kOnce) __builtin_nontemporal_store(v, q);
    else *q = v;
}
template <bool kOnce>
__device__ __forceinline__ void write(uint32_t* p, words4 v) {
    words4_at4* q = reinterpret_cast<words4_at4*>(p);
    if (kOnce) __builtin_nontemporal_store(v, q);
    else *q = v;
}

// Eight channels as they stand in memory.
template <int kBf16>
struct Raw {
    words4 q[kBf16 ? 1 : 2];
    __device__ __forceinline__ float get(int i) const {
        if (kBf16) {
            const uint32_t w = q[0][i >> 1];
            return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
        }
        return __uint_as_float(q[i >> 2][i & 3]);
    }
};

// The eight channels from element `at` of a row that has n >= 1 left from there
// (channels behind the row's end: 0).  kWhole: n is at least eight.  kOnce: rows that
// nothing reads again soon (non-temporal, whole eights only).
template <int kBf16, bool kWhole = false, bool kOnce = false>
__device__ __forceinline__ Raw<kBf16> load(const void* row, int64_t at, int64_t n) {
    Raw<kBf16> r;
    if (kBf16) {
        const uint16_t* p = (const uint16_t*)row + at;
        if (kWhole || n >= kPer) {
            r.q[0] = read<kOnce>(p);
        } else {
            uint32_t v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = i < n ? (uint32_t)p[i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) r.q[0][i] = v[2 * i] | (v[2 * i + 1] << 16);
        }
    } else {
        const uint32_t* p = (const uint32_t*)row + at;
        if (kWhole || n >= kPer) {
            r.q[0] = read<kOnce>(p);
            r.q[1] = read<kOnce>(p + 4);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) r.q[i >> 2][i & 3] = i < n ? p[i] : 0u;
        }
    }
    return r;
}

typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_bits(float a, float b) {
    const bf16_pair v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
// Eight fp32 values in the type's form, each rounded once.
template <int kBf16>
__device__ __forceinline__ Raw<kBf16> pack(const float* v) {
    Raw<kBf16> r;
    if (kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.q[0][i] = bf16_bits(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) r.q[i >> 2][i & 3] = __float_as_uint(v[i]);
    }
    return r;
}
template <int kBf16, bool kWhole = false, bool kOnce = false>
__device__ __forceinline__ void store(void* row, int64_t at, int64_t n, const Raw<kBf16>& r) {
    if (kBf16) {
        uint16_t* p = (uint16_t*)row + at;
        if (kWhole || n >= kPer) {
            write<kOnce>(p, r.q[0]);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i < n) p[i] = (uint16_t)(r.q[0][i >> 1] >> (16 * (i & 1)));
        }
    } else {
        uint32_t* p = (uint32_t*)row + at;
        if (kWhole || n >= kPer) {
            write<kOnce>(p, r.q[0]);
            write<kOnce>(p + 4, r.q[kBf16 ? 0 : 1]);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i < n) p[i] = r.q[i >> 2][i & 3];
        }
    }
}

// Sums and maxima over the kL lanes (8 .. 64, aligned groups) that share a row, the
// same bits in each of them: within 16 lanes by DPP moves, across them by gfx950's
// swaps of rows and halves.  Every lane is active.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp<kCtrl>((uint32_t)b), hi = dpp<kCtrl>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, lo | hi << 32);
}
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp<kCtrl>(__float_as_uint(v)));
}
struct Two {
    uint32_t a, b;
};
template <int kSpan>                         // 16: rows 0|1 and 2|3; 32: halves
__device__ __forceinline__ Two both(uint32_t v) {
    const auto r = kSpan == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                               : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return {(uint32_t)r[0], (uint32_t)r[1]};
}
template <int kSpan>
__device__ __forceinline__ double both_sum(double v) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    const Two lo = both<kSpan>((uint32_t)w), hi = both<kSpan>((uint32_t)(w >> 32));
    return __builtin_bit_cast(double, (uint64_t)lo.a | (uint64_t)hi.a << 32) +
           __builtin_bit_cast(double, (uint64_t)lo.b | (uint64_t)hi.b << 32);
}
template <int kSpan>
__device__ __forceinline__ float both_sum(float v) {
    const Two t = both<kSpan>(__float_as_uint(v));
    return __uint_as_float(t.a) + __uint_as_float(t.b);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;
template <int kL, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
    if (kL >= 2) v += dpp<kXor1>(v);
    if (kL >= 4) v += dpp<kXor2>(v);
    if (kL >= 8) v += dpp<kMirror8>(v);
    if (kL >= 16) v += dpp<kMirror16>(v);
    if (kL >= 32) v = both_sum<16>(v);
    if (kL >= 64) v = both_sum<32>(v);
    return v;
}
template <typename T>
__device__ __forceinline__ T larger(T a, T b) {
    return a > b ? a : b;
}
template <int kL>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if (kL >= 2) v = larger(v, dpp<kXor1>(v));
    if (kL >= 4) v = larger(v, dpp<kXor2>(v));
    if (kL >= 8) v = larger(v, dpp<kMirror8>(v));
    if (kL >= 16) v = larger(v, dpp<kMirror16>(v));
    if (kL >= 32) {
        const Two t = both<16>(v);
        v = larger(t.a, t.b);
    }
    if (kL >= 64) {
        const Two t = both<32>(v);
        v = larger(t.a, t.b);
    }
    return v;
}

// How the rows' length goes into eights: whole ones only; the last one partial; less
// than one.
enum Cut { kEven = 0, kOdd = 1, kTiny = 2 };
inline Cut cut_of(int64_t H) { return H % kPer == 0 ? kEven : (H < kPer ? kTiny : kOdd); }

// The eight channels of a thread in a row of len channels: elements at .. at + 7, of
// which those from `from` on are its own.  The row's last, partial eight (kOdd) start
// earlier and share channels with the eight before: what both compute is the same, so
// both may store it once no other thread reads what was there any more (else store_own),
// and sums leave out what is not the thread's own.  (Reading and storing a partial eight
// element by element takes a row's work-group three latencies more, 16384 x 1001 bf16
// 21.3 us against 15.9, 8192 x 5001 93 against 79.)
struct Piece {
    int at, from, n;                         // n: how many there are, 0 .. 8
};
template <int kCut>
__device__ __forceinline__ Piece piece(int c, int len) {
    if (c >= len) return {0, 0, 0};
    if (kCut == kTiny) return {c, 0, len - c};
    if (kCut == kEven || len - c >= kPer) return {c, 0, kPer};
    return {len - kPer, c - (len - kPer), kPer};
}
// The piece's own channels alone.
template <int kBf16>
__device__ __forceinline__ void store_own(void* row, const Piece& p, const Raw<kBf16>& r) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i < p.from || i >= p.n) continue;
        if (kBf16) ((uint16_t*)row)[p.at + i] = (uint16_t)(r.q[0][i >> 1] >> (16 * (i & 1)));
        else ((uint32_t*)row)[p.at + i] = r.q[kBf16 ? 0 : i >> 2][i & 3];
    }
}

// Element address of a row, whatever the type.
template <int kBf16>
__device__ __forceinline__ const void* row_at(const void* base, int64_t element) {
    return (const char*)base + element * (kBf16 ? 2 : 4);
}
template <int kBf16>
__device__ __forceinline__ void* row_at(void* base, int64_t element) {
    return (char*)base + element * (kBf16 ? 2 : 4);
}

// ------------------------------------------------------------------ host --
inline bool ok_type(int t) { return t == QUADS_OUT_F32 || t == QUADS_OUT_BF16; }
inline bool ok_opt4(const void* p) { return p == nullptr || ok_ptr4(p); }
constexpr int64_t kMaxH = (int64_t)1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

}  // namespace block
}  // namespace quads
