// Shared by the kernels of the layer around the experts (quads_block.h): rows
// of channels in bf16 or fp32, read and written eight channels at a time.
//
// A row may start at any element (odd lengths, row strides of the caller's):
// the eight channels of a thread are one 16-byte access (bf16) or two (fp32)
// at whatever address they have, which gfx950 takes; only a row's last, partial
// eight go element by element.
#pragma once

#include "common.h"
#include "../../include/quads_block.h"

namespace quads {
namespace block {

constexpr int kPer = 8;                      // channels per access

typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef words4 words4_at2 __attribute__((aligned(2)));
typedef words4 words4_at4 __attribute__((aligned(4)));
typedef uint32_t words2 __attribute__((ext_vector_type(2)));

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
// (channels behind the row's end: 0).
template <int kBf16>
__device__ __forceinline__ Raw<kBf16> load(const void* row, int64_t at, int64_t n) {
    Raw<kBf16> r;
    if (kBf16) {
        const uint16_t* p = (const uint16_t*)row + at;
        if (n >= kPer) {
            r.q[0] = *reinterpret_cast<const words4_at2*>(p);
        } else {
            uint32_t v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = i < n ? (uint32_t)p[i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) r.q[0][i] = v[2 * i] | (v[2 * i + 1] << 16);
        }
    } else {
        const uint32_t* p = (const uint32_t*)row + at;
        if (n >= kPer) {
            r.q[0] = *reinterpret_cast<const words4_at4*>(p);
            r.q[1] = *reinterpret_cast<const words4_at4*>(p + 4);
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
template <int kBf16>
__device__ __forceinline__ void store(void* row, int64_t at, int64_t n, const Raw<kBf16>& r) {
    if (kBf16) {
        uint16_t* p = (uint16_t*)row + at;
        if (n >= kPer) {
            *reinterpret_cast<words4_at2*>(p) = r.q[0];
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i < n) p[i] = (uint16_t)(r.q[0][i >> 1] >> (16 * (i & 1)));
        }
    } else {
        uint32_t* p = (uint32_t*)row + at;
        if (n >= kPer) {
            *reinterpret_cast<words4_at4*>(p) = r.q[0];
            *reinterpret_cast<words4_at4*>(p + 4) = r.q[kBf16 ? 0 : 1];
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i < n) p[i] = r.q[i >> 2][i & 3];
        }
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
constexpr int64_t kMaxH = (int64_t)1 << 26;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

}  // namespace block
}  // namespace quads
