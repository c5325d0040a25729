// W4A16 grouped product for few rows per expert (include/quads_head.h): bf16
// activations times NVFP4 weights, arXiv 2607.15810, Eq. (12).
//
//   Y[p, n] = s_tW[e] sum_j x[row(p), j] v_w[n, j] s_b[n, j / 16]
//
// What bounds it is the weights' stream from HBM, 0.5625 bytes per weight, so
// every weight is loaded once per 16 kRt rows, straight into the registers
// of the wave that uses it, as wide as it lies, and multiplied on the matrix
// cores, where up to 16 rows cost no more than one.
//
// Operands.  A weight's v * s_b has at most 6 significant bits and lies in
// [2^-10, 2688]: exact in fp16, converted by the hardware's fp4 convert and
// one packed multiply per two weights.  bf16 has no packed multiply, so the
// activations are brought to fp16 instead: every 512 channels of a row are
// scaled by the power of two that puts their largest magnitude in [2^14,
// 2^15), exact for every activation down to 2^-28 of that largest one (below
// it the error is at most 2^-28 of the largest), and the scale goes into the
// fp32 total when the matrix cores' accumulator is added to it, every 512
// channels (gfx950's fp16 MFMA rounds once per 8 products: 64 roundings).
//
// Layout.  A work-group has kWaves waves; a wave owns two tiles of 16
// features (SwiGLU: 16 gate features and the 16 up features that belong to
// them) and streams them in blocks of 512 channels.  Lane (r, h) = (lane %
// 16, lane / 16) holds feature r: of each 128-channel chunk the 32 codes from
// channel 32 h on (one 16-byte load, 64 contiguous bytes per feature and
// load), and step j of a chunk multiplies the lane's codes 8 j .. 8 j + 7, so
// the channels of the four h interleave; the activations are read from LDS in
// the same order.  When a block has been multiplied the next one's loads go
// out together, 256 contiguous bytes of every feature: spread out, chunk by
// chunk as each was consumed, they asked for the two halves of a 128-byte line
// at different times and cost 6% (1 x 2048 x 262144: 63.8 against 59.5 us; a
// read of the same bytes in order takes 59.8).  The other waves of the SIMD
// multiply meanwhile.
//   The block scales of 512 channels of a feature are 32 bytes: lane (r, h)
// loads the 8 of chunk h, and the four lanes of a feature exchange them in
// registers (row swaps), so that each has its two of every chunk.
//   The activations, few and read by every wave, are in LDS: all of a unit's
// channels, brought once, where they fit (K <= 4608 for 16 rows, 9216 for 8), else
// as many blocks as do, again for every step.  A wave then takes its features
// alone, and there are at most outputs / 128 work-groups, too few for the GPU at
// ordinary N: 16 x 4608 x 4096 takes 16.5 us and 16 x 5120 x 4096 35, 9 x 8192 x
// 4096 19 and 10 x 8192 x 4096 50, 16 x 7168 x 7168 48 (0.6 TB/s).
//
// Work-groups are resident ones, as many as the GPU holds: a unit (up to 16 kRt
// rows of an expert) has `slabs` of them, and each takes an equal range of its
// features, in steps of two tiles per slot of kw waves; the kw waves of a slot
// share its tiles, each taking every kw-th block, and their totals are added
// in LDS in wave order.  The ranges are even to 4 features: lanes past a
// slot's last feature load nothing, so no work-group streams more than its
// share (whole tiles per wave, one or two of them, left a third of the waves
// idle at the end: 13 x 2048 x 100003 took 36 us, 1 x 4096 x 150000 84 us).
#include "common.h"
#include "gemm_tiles.h"
#include "../../include/quads_head.h"

namespace quads {
namespace w4a16 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kChunk = 128;                    // channels per 16-byte load
constexpr int kBlk = 512;                      // channels per block
constexpr int kStage = 4;                      // activation loads in flight per wave
constexpr int kLds = 160 << 10;                // LDS bytes of a CU
constexpr int kCus = 256;
constexpr int kHeld = 4;                       // experts' offsets per lane kept in registers

struct Args {
    const uint16_t* x; const int32_t* row_token; int rows; int K;
    const uint8_t* w_nib; const uint8_t* w_scale; const float* w_ts; const int32_t* offsets;
    int E; int N;
    int out_bf16; void* out;
    int kw;                                    // waves per slot
    int slabs;                                 // work-groups per unit of rows
    int steps;                                 // of the largest slot
    int step;                                  // features per step
    int sb;                                    // blocks of activations in LDS at once
    int rcap;                                  // rows of LDS
};

// Unaligned wide loads: a feature's codes start at a multiple of 8 bytes, its
// scales anywhere.
struct __attribute__((packed)) Bytes16 { u32x4 v; };
struct __attribute__((packed)) Bytes8 { u32x2 v; };

// 8 codes (one dword) times a block scale -> 8 exact fp16 values.
__device__ __forceinline__ f16x8 cvt8(uint32_t w, _Float16 s) {
    const f16x2 s2 = {s, s};
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s2;
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s2;
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s2;
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s2;
    return (f16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A feature's codes of chunk `cc` for the lane: 32 from channel 128 cc + 32 h
// on, at the uniform base `at` (the tile's first feature) plus the lane's
// `off`.  Codes past K read as 0; a lane that is not `ok` loads nothing.
__device__ __forceinline__ uint4 load_codes(const uint8_t* at, uint32_t off, int cc, int h, int K,
                                            bool ok) {
    const uint8_t* p = at + (int64_t)cc * (kChunk / 2);
    if ((cc + 1) * kChunk <= K) {
        u32x4 v = {0, 0, 0, 0};
        if (ok) v = reinterpret_cast<const Bytes16*>(p + off)->v;
        return make_uint4(v.x, v.y, v.z, v.w);
    }
    const int k = cc * kChunk + 32 * h;
    u32x2 lo = {0, 0}, hi = {0, 0};
    if (ok && k < K) lo = reinterpret_cast<const Bytes8*>(p + off)->v;
    if (ok && k + 16 < K) hi = reinterpret_cast<const Bytes8*>(p + off + 8)->v;
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
// A feature's scales of chunk 4 b + h (8 bytes); 0 past K.
__device__ __forceinline__ u32x2 load_scales(const uint8_t* at, uint32_t off, int b, int h, int K,
                                             bool ok) {
    const int cc = 4 * b + h;
    const uint8_t* p = at + (int64_t)b * (kBlk / kBlock) + (off + 8u * h);
    u32x2 v = {0, 0};
    if (!ok) return v;
    if ((cc + 1) * kChunk <= K) {
        v = reinterpret_cast<const Bytes8*>(p)->v;
    } else {
        const int n = K / kBlock - cc * (kChunk / kBlock);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
    return v;
}

// From the scales of chunk h to the lane's own two of every chunk (fp8 pairs
// in the low 16 bits): lane h's pair of chunk c is bytes 2 h, 2 h + 1 of what
// the lane of chunk c loaded.
__device__ __forceinline__ void own_scales(u32x2 v, int h, uint32_t s[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.y, false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);   // chunks 0, 1
    const auto f = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);   // chunks 2, 3
    const int sh = 16 * (h & 1);
    s[0] = e[0] >> sh;
    s[1] = e[1] >> sh;
    s[2] = f[0] >> sh;
    s[3] = f[1] >> sh;
}

// Dynamic LDS: [rcap][sb * 1024 + 16] bytes of fp16 activations, [rcap][sb]
// fp32 scales of their blocks, then the totals of each slot's waves but the
// first.
template <int kEpi, int kRt>
__global__ __launch_bounds__(kThreads, 4) void k_w4a16(Args g) {
    constexpr bool swiglu = kEpi == QUADS_EPI_SWIGLU;
    constexpr int kRows = 16 * kRt;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, h = lane >> 4;
    const int slab = (int)(blockIdx.x % (unsigned)g.slabs);
    const int rank = (int)(blockIdx.x / (unsigned)g.slabs);

    // the unit of this rank: kRows rows of an expert, in expert order.  Lane l
    // counts the units of experts l*per .. l*per + per - 1, a scan finds the
    // lane, the lane finds the expert.  Up to kHeld experts a lane keeps the
    // offsets in registers, loaded together: the weights wait for them.
    int e = 0, p0 = kRows * rank, cnt = g.rows - p0;
    if (g.offsets) {
        const int per = (g.E + 63) / 64;
        const int e0 = lane * per < g.E ? lane * per : g.E;
        const int e1 = e0 + per < g.E ? e0 + per : g.E;
        int held[kHeld + 1];
#pragma unroll
        for (int i = 0; i <= kHeld; ++i) held[i] = g.offsets[e0 + i < g.E ? e0 + i : g.E];
        int na = 0;
        if (per <= kHeld) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                na += e0 + i < e1 ? (held[i + 1] - held[i] + kRows - 1) / kRows : 0;
        } else {
            for (int x = e0; x < e1; ++x)
                na += (g.offsets[x + 1] - g.offsets[x] + kRows - 1) / kRows;
        }
        const int inc = wave_incl_add(na);
        if (rank >= __builtin_amdgcn_readlane(inc, 63)) return;
        int found = -1, from = 0, to = 0;
        int rr = rank - (inc - na);
        if (rr >= 0 && rank < inc) {
            if (per <= kHeld) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    const int u = e0 + i < e1 ? (held[i + 1] - held[i] + kRows - 1) / kRows : 0;
                    if (found < 0 && rr < u) {
                        found = e0 + i;
                        from = held[i] + kRows * rr;
                        to = held[i + 1];
                    }
                    rr -= u;
                }
            } else {
                for (int x = e0; x < e1; ++x) {
                    const int u = (g.offsets[x + 1] - g.offsets[x] + kRows - 1) / kRows;
                    if (rr < u) {
                        found = x;
                        from = g.offsets[x] + kRows * rr;
                        to = g.offsets[x + 1];
                        break;
                    }
                    rr -= u;
                }
            }
        }
        const int src = __ffsll(__ballot(found >= 0)) - 1;
        e = __builtin_amdgcn_readlane(found, src);
        p0 = __builtin_amdgcn_readlane(from, src);
        cnt = __builtin_amdgcn_readlane(to, src) - p0;
    }
    if (cnt <= 0) return;
    const int nr = cnt < kRows ? cnt : kRows;
    // lane l: the activation row of the unit's row l
    int token = 0;
    if (lane < nr) token = g.row_token ? g.row_token[p0 + lane] : p0 + lane;

    // the slot's output features [lo, hi), taken g.step at a time
    const int nout = swiglu ? g.N / 2 : g.N;
    const int wk = wave % g.kw;
    const int slots = kWaves / g.kw;
    const int64_t slot = (int64_t)slab * slots + wave / g.kw, all = (int64_t)g.slabs * slots;
    const int64_t quads_n = (nout + 3) / 4;
    const int lo = __builtin_amdgcn_readfirstlane((int)(4 * (quads_n * slot / all)));
    const int hi =
        __builtin_amdgcn_readfirstlane(min(nout, (int)(4 * (quads_n * (slot + 1) / all))));
    const int nblk = (g.K + kBlk - 1) / kBlk;
    // each tile's first feature (of the weight rows), g.step rows further per
    // step, and how many of its features there are; the lane's offset from it
    const uint8_t* nib[2];
    const uint8_t* sc[2];
    int left[2], most[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int f = lo + (swiglu ? 0 : 16 * q);
        const int64_t row = (int64_t)e * g.N + f + (swiglu ? q * nout : 0);
        nib[q] = g.w_nib + row * (g.K / 2);
        sc[q] = g.w_scale + row * (g.K / kBlock);
        left[q] = hi - f;
        most[q] = g.step - (swiglu ? 0 : 16 * q);
    }
    const uint32_t nib_off = (uint32_t)r * (g.K / 2) + 16 * h, sc_off = (uint32_t)r * (g.K / kBlock);
    const int64_t nib_step = (int64_t)g.step * (g.K / 2), sc_step = (int64_t)g.step * (g.K / kBlock);

    uint4 code[2][4];
    u32x2 scale[2];
    auto load = [&](int b) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const bool ok = r < min(left[q], most[q]) && b < nblk;
            scale[q] = load_scales(sc[q], sc_off, b, h, g.K, ok);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                code[q][c] = load_codes(nib[q], nib_off, 4 * b + c, h, g.K, ok);
        }
    };
    load(wk);

    const int stride = g.sb * 2 * kBlk + 16;
    float* xscale = (float*)(lds + (size_t)g.rcap * stride);
    f32x4* part = reinterpret_cast<f32x4*>(
        lds + (((size_t)g.rcap * (stride + 4 * g.sb) + 15) & ~(size_t)15));
    int xrow[kRt];
#pragma unroll
    for (int t = 0; t < kRt; ++t) xrow[t] = 16 * t + r < nr ? 16 * t + r : 0;
    const float ts = g.w_ts[e];

    for (int st = 0; st < g.steps; ++st) {
        f32x4 tot[2][kRt];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int t = 0; t < kRt; ++t) tot[q][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = 0; s0 < nblk; s0 += g.sb) {
            const int sb = nblk - s0 < g.sb ? nblk - s0 : g.sb;
            if (st == 0 || g.sb < nblk) {
                if (st > 0 || s0 > 0) __syncthreads();
                // activations of blocks s0 .. s0 + sb - 1: a wave per (row,
                // block), kStage of them requested together
                for (int i0 = wave; i0 < nr * sb; i0 += kStage * kWaves) {
                    uint4 v[kStage];
#pragma unroll
                    for (int a = 0; a < kStage; ++a) {
                        const int i = i0 + a * kWaves;
                        v[a] = make_uint4(0, 0, 0, 0);
                        if (i < nr * sb) {
                            const int k = (s0 + i % sb) * kBlk + 8 * lane;
                            const int64_t src = __builtin_amdgcn_readlane(token, i / sb);
                            if (k < g.K)
                                v[a] = *reinterpret_cast<const uint4*>(g.x + src * g.K + k);
                        }
                    }
#pragma unroll
                    for (int a = 0; a < kStage; ++a) {
                        const int i = i0 + a * kWaves;
                        if (i >= nr * sb) break;
                        const int row = i / sb, b = i % sb;
                        const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
                        uint32_t m = 0;
#pragma unroll
                        for (int u = 0; u < 4; ++u) m = pk_max_u16(m, w[u] & 0x7FFF7FFFu);
                        m = wave_max_u32(umax32(m >> 16, m & 0xFFFFu));
                        // 2^(141 - ex) with ex the exponent of the largest
                        // magnitude; blocks below 2^-112 take the largest
                        // power with a normal inverse
                        uint32_t ex = m >> 7;
                        ex = ex < 15u ? 15u : ex;
                        const float up = __uint_as_float((268u - ex) << 23);
                        f16x8 y;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            y[2 * u] = (_Float16)(__uint_as_float(w[u] << 16) * up);
                            y[2 * u + 1] = (_Float16)(__uint_as_float(w[u] & 0xFFFF0000u) * up);
                        }
                        *reinterpret_cast<f16x8*>(lds + row * stride + 2 * (b * kBlk + 8 * lane)) =
                            y;
                        if (lane == 0) xscale[row * g.sb + b] = __uint_as_float((ex - 14u) << 23);
                    }
                }
                __syncthreads();
            }
            // the wave's blocks among them (sb is a multiple of kw, or all)
            for (int b = s0 + wk; b < s0 + sb; b += g.kw) {
                f32x4 acc[2][kRt];
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int t = 0; t < kRt; ++t) acc[q][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
                uint32_t own[2][4];
#pragma unroll
                for (int q = 0; q < 2; ++q) own_scales(scale[q], h, own[q]);
                const char* xb = lds + 2 * ((b - s0) * kBlk + 32 * h);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    f16x2 s[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        s[q] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(own[q][c], 1.0f, false);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f16x8 xf[kRt];
#pragma unroll
                        for (int t = 0; t < kRt; ++t)
                            xf[t] = *reinterpret_cast<const f16x8*>(xb + xrow[t] * stride +
                                                                    2 * (kChunk * c + 8 * j));
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint4& w = code[q][c];
                            const uint32_t x = j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
                            const f16x8 wf = cvt8(x, s[q][j >> 1]);
#pragma unroll
                            for (int t = 0; t < kRt; ++t)
                                acc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                    wf, xf[t], acc[q][t], 0, 0, 0);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                // what follows this block: the wave's next one, or its first
                // of the next step
                const bool turn = b + g.kw >= nblk;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (turn) {
                        nib[q] += nib_step;
                        sc[q] += sc_step;
                        left[q] -= g.step;
                    }
                load(turn ? wk : b + g.kw);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < kRt; ++t) {
                    const float f = xscale[xrow[t] * g.sb + b - s0];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            tot[q][t][u] = __builtin_fmaf(acc[q][t][u], f, tot[q][t][u]);
                }
            }
        }

        // totals of the slot's waves: into LDS, added in wave order
        if (g.kw > 1) {
            if (st > 0) __syncthreads();
            if (wk > 0) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int t = 0; t < kRt; ++t)
                        part[(((wave - 1) * 2 + q) * kRt + t) * 64 + lane] = tot[q][t];
            }
            __syncthreads();
            if (wk > 0) continue;
            for (int w = 1; w < g.kw; ++w)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int t = 0; t < kRt; ++t)
                        tot[q][t] += part[(((wave + w - 1) * 2 + q) * kRt + t) * 64 + lane];
        }

        // lane (r, h) holds row 16 t + r of features 4 h .. 4 h + 3 of each tile
        const int end = min(hi, lo + (st + 1) * g.step);
#pragma unroll
        for (int t = 0; t < kRt; ++t) {
            const bool have = 16 * t + r < nr;
            const int64_t o = (int64_t)(p0 + 16 * t + r) * nout;
#pragma unroll
            for (int q = 0; q < (swiglu ? 1 : 2); ++q) {
                const int n = lo + st * g.step + 16 * q + 4 * h;
                float y[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    y[u] = tot[q][t][u] * ts;
                    if (swiglu) y[u] = silu_mul(y[u], tot[1][t][u] * ts);
                }
                if (!have || n >= end) continue;
                if (g.out_bf16) {
                    uint16_t* a = (uint16_t*)g.out + o + n;
                    const uint32_t p01 = v2::pk_bf16(y[0], y[1]), p23 = v2::pk_bf16(y[2], y[3]);
                    if (nout % 4 == 0) {
                        *reinterpret_cast<uint2*>(a) = make_uint2(p01, p23);
                    } else {
                        const uint32_t b4[4] = {p01, p01 >> 16, p23, p23 >> 16};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (n + u < end) a[u] = (uint16_t)b4[u];
                    }
                } else {
                    float* a = (float*)g.out + o + n;
                    if (nout % 4 == 0) {
                        *reinterpret_cast<float4*>(a) = make_float4(y[0], y[1], y[2], y[3]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (n + u < end) a[u] = y[u];
                    }
                }
            }
        }
    }
}

template <int kEpi, int kRt>
int launch(Args g, hipStream_t st) {
    constexpr int kRows = 16 * kRt;
    constexpr int kStep = kEpi == QUADS_EPI_SWIGLU ? 16 : 32;
    const int nout = kEpi == QUADS_EPI_SWIGLU ? g.N / 2 : g.N;
    const int64_t units = g.offsets ? (int64_t)(g.E < g.rows ? g.E : g.rows) + g.rows / kRows
                                    : ((int64_t)g.rows + kRows - 1) / kRows;
    // units that have work, as far as the host can tell
    int64_t live = units;
    if (g.offsets) {
        live = g.E < g.rows ? g.E : g.rows;
        if (live < g.rows / kRows) live = g.rows / kRows;
    }
    const int nblk = (g.K + kBlk - 1) / kBlk;
    g.rcap = g.rows < kRows ? g.rows : kRows;
    // All channels in LDS, two work-groups a CU if that fits, else one; the
    // waves of a slot then share out its blocks.  Else a wave takes its tiles
    // alone, and the activations are brought anew for every step.
    const size_t row = 2 * kBlk + 4, part = (size_t)2 * kRt * 64 * 16;
    g.kw = 1;
    while (g.kw < kWaves && 2 * g.kw <= nblk) g.kw *= 2;
    const size_t join = g.kw > 1 ? (kWaves - 1) * part : 0;
    auto blocks = [&](size_t bytes) {
        return bytes < 1024 ? 0 : ((int64_t)((bytes - 16) / g.rcap) - 16) / (int64_t)row;
    };
    const size_t two = kLds / 2, one = kLds - 1024;
    bool pairs = true;
    if (blocks(two - join) >= nblk) {
        g.sb = nblk;
    } else if (blocks(one - join) >= nblk) {
        g.sb = nblk;
        pairs = false;
    } else {
        g.kw = 1;
        g.sb = (int)blocks(two);
        if (g.sb > nblk) g.sb = nblk;
    }
    // as many work-groups as are resident, but at least 16 features per slot
    const int slots = kWaves / g.kw;
    int64_t slabs = (pairs ? 2 : 1) * kCus / live;
    const int64_t most = ((int64_t)nout + 16 * slots - 1) / (16 * slots);
    if (slabs > most) slabs = most;
    if (slabs < 1) slabs = 1;
    g.slabs = (int)slabs;
    const int64_t quads_n = (nout + 3) / 4, share = (quads_n + slabs * slots - 1) / (slabs * slots);
    // steps of equal size (multiples of 4 features)
    g.steps = (int)((4 * share + kStep - 1) / kStep);
    g.step = (int)(4 * ((share + g.steps - 1) / g.steps));
    size_t bytes = (g.rcap * (16 + g.sb * row) + 15) & ~(size_t)15;
    if (g.kw > 1) bytes += (kWaves - 1) * part;
    hipLaunchKernelGGL((k_w4a16<kEpi, kRt>), dim3((unsigned)(slabs * units)), dim3(kThreads),
                       bytes, st, g);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

// Rows per unit: 16; 32, so that the weights are read half as often, where
// experts have that many, all channels of 32 rows fit in LDS (K <= 2048: one
// work-group a CU) and the weights are larger than the 32 MB of L2, which
// otherwise serves the second read.  In us with 16 / 32 rows: 40 x 2048 x
// 32768 30.6 / 28.0; gate/up of 128 experts of 1536 x 2048, top 8, 256 tokens
// 71 / 62, 128 tokens 52 / 60; 16 such experts, 64 tokens 29 / 36; 64 x 4096 x
// 4096 17.6 / 38.  64 rows were never better than both.  (The form of 32 rows
// spills 5 registers, with SwiGLU 1: stored before the loop over the steps, read
// back at a step's results.)  Either way a unit of rows decodes the weights for
// itself after it has brought all of its activations, so that 17 to 64 rows of a
// matrix take 3 to 9 times what their bytes do.
template <int kEpi>
int dispatch(const Args& g, hipStream_t st) {
    const double bytes = 0.5625 * g.E * g.N * g.K;
    const bool many = g.offsets ? g.rows / g.E >= 16 : g.rows > 16;
    if (many && g.K <= 2048 && bytes > 32.0 * (1 << 20)) return launch<kEpi, 2>(g, st);
    return launch<kEpi, 1>(g, st);
}

}  // namespace w4a16
}  // namespace quads

using namespace quads;

// The product needs none; the pair of calls is the library's form.
extern "C" size_t quads_moe_w4a16_gemv_ws(int64_t rows, int64_t K, int32_t E, int64_t N) {
    (void)rows; (void)K; (void)E; (void)N;
    return 0;
}

extern "C" int quads_moe_w4a16_gemv(const uint16_t* x, const int32_t* row_token, int64_t rows,
                                    int64_t K, const uint8_t* w_nib, const uint8_t* w_scale,
                                    const float* w_ts, const int32_t* offsets, int32_t E,
                                    int64_t N, int epilogue, int out_dtype, void* out, void* ws,
                                    size_t ws_bytes, void* stream) {
    if (rows < 0 || rows >= ((int64_t)1 << 24) || K <= 0 || K % kBlock || K >= ((int64_t)1 << 26) ||
        E < 1 || E > 4096 || N < 1 || N >= ((int64_t)1 << 30))
        return QUADS_ESHAPE;
    if (epilogue != QUADS_EPI_NONE && epilogue != QUADS_EPI_SWIGLU) return QUADS_EINVAL;
    if (out_dtype != QUADS_OUT_F32 && out_dtype != QUADS_OUT_BF16) return QUADS_EINVAL;
    if (epilogue == QUADS_EPI_SWIGLU && out_dtype != QUADS_OUT_BF16) return QUADS_EINVAL;
    if (epilogue == QUADS_EPI_SWIGLU && N % 2) return QUADS_ESHAPE;
    if (offsets == nullptr && E != 1) return QUADS_EINVAL;
    if (rows == 0) return QUADS_OK;
    if ((offsets != nullptr && !ok_ptr4(offsets)) || (row_token != nullptr && !ok_ptr4(row_token)))
        return QUADS_EINVAL;
    if (!ok_ptr(x) || !ok_ptr(w_nib) || !ok_ptr(w_scale) || !ok_ptr4(w_ts) || !ok_ptr(out))
        return QUADS_EINVAL;
    (void)ws; (void)ws_bytes;
    w4a16::Args g{};
    g.x = x; g.row_token = row_token; g.rows = (int)rows; g.K = (int)K;
    g.w_nib = w_nib; g.w_scale = w_scale; g.w_ts = w_ts; g.offsets = offsets;
    g.E = (int)E; g.N = (int)N; g.out_bf16 = out_dtype == QUADS_OUT_BF16; g.out = out;
    return epilogue == QUADS_EPI_SWIGLU ? w4a16::dispatch<QUADS_EPI_SWIGLU>(g, (hipStream_t)stream)
                                        : w4a16::dispatch<QUADS_EPI_NONE>(g, (hipStream_t)stream);
}
