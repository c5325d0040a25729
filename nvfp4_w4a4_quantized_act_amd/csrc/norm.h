// Shared by the norm's kernels (norm.hip) and its gradient's (norm_grad.hip).
//
//   h = RN(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = h r w
//   n = h r,  c = mean(n w g),  dh = g_sum + r (w g - n c),  dw = sum_t g n
//
// h^2 of bf16 or fp32 numbers and their sum are held in fp64: the sum cannot
// overflow, and the 8-bit output's codes are decided by comparisons of y with the
// format's borders, which fp32 statistics would move.
#pragma once

#include "block.h"

namespace quads {
namespace norm {

using namespace block;

constexpr int kNone = 2;                     // no residual

// Sum over a work-group of up to 16 waves (one barrier), in every thread.  s_part: two
// sets of one number per wave, taken in turn by calls that follow one another (`set`
// 0, 1, 0, ..): a wave is past the barrier of the call between when it writes a set
// again, and so every wave has read it.
constexpr int kMaxWaves = 16;
__device__ __forceinline__ double group_sum(double v, double (*s_part)[kMaxWaves], int set) {
    v = lanes_sum<64>(v);
    if ((threadIdx.x & 63) == 0) s_part[set][threadIdx.x >> 6] = v;
    __syncthreads();
    const int i = threadIdx.x & (kMaxWaves - 1);
    return lanes_sum<kMaxWaves>(i < (int)(blockDim.x >> 6) ? s_part[set][i] : 0.0);
}

// Eight channels of the weight in either type; 1 without one.
__device__ __forceinline__ void load_weight(const void* weight, int dtype, int64_t c, int64_t n,
                                            float* w) {
    if (dtype == QUADS_OUT_BF16) {
        const Raw<1> r = load<1>(weight, c, n);
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = r.get(i);
    } else if (dtype == QUADS_OUT_F32) {
        const Raw<0> r = load<0>(weight, c, n);
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = r.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = 1.0f;
    }
}
constexpr int kNoWeight = -1;

inline int check_sizes(int64_t T, int64_t H, int64_t ld) {
    if (T < 0 || T >= ((int64_t)1 << 31) || H < 1 || H >= kMaxH) return QUADS_ESHAPE;
    return ld < H || ld >= kMaxStride ? QUADS_ESHAPE : QUADS_OK;
}
// r is held in fp32 where it is not in fp64.
inline bool ok_eps(double eps) { return eps >= 1e-70 && eps <= 1e70; }

}  // namespace norm
}  // namespace quads
