// Tokens in packed (expert) order and back, and the gradient of the way back.  The MoE
// combine of quads.h is the way back with weights and fp32 output.
//
//   sort     out[pos[t, s]] = x[t]
//   unsort   out[t] = sum_s w[t, s] y[pos[t, s]]
//   gradient dy[pos[t, s]] = w[t, s] g[t],  dw[t, s] = <g[t], y[pos[t, s]]>
//
// Copies of rows: HBM bounds them.  Both directions go by token: the token's own
// row is then read (or written) once, and what is many rows, the packed side,
// once too, whole rows of it at places of its own.
#include "block.h"

#include <type_traits>

namespace quads {
namespace sorting {

using namespace block;

constexpr int kMaxTopk = 64;

struct Args {
    const void* a;                           // x, y or g
    const void* y;                           // of the gradient
    void* out;                               // packed rows, token rows, or dy
    float* dw;
    int64_t T, H, ld, rows;                  // ld: of x, and of y and out on the way back
    int topk, per;                           // per: slots of a work-group of the gradient
    const int32_t* slot_of;                  // [rows], where rows without a slot become 0
    int64_t slots;                           // of the whole call
    unsigned groups;                         // work-groups with tokens; behind them zero_rest's
};

// Rows without a slot become 0 in one of two ways.  Up to kFillBytes every row is zeroed
// first; beyond, that would write most of them twice, and those without a slot are found
// with an inverse of pos that nobody clears: slot_of[pos[i]] = i for every slot i, and
// whatever the memory held elsewhere; row p has a slot if its entry is some i whose pos is
// p.  Device time of the sort, all rows first / found, rows for 5/4 of the slots: 64 x 2048,
// top 8, bf16 5.2 us / 8.5, 1000 x 1000, top 4, bf16 6.7 / 8.7, 4096 x 2048, top 8, bf16
// 45.2 / 40.2, 16384 x 4096, top 8, bf16 385 / 318.
constexpr int64_t kFillBytes = (int64_t)64 << 20;
__global__ __launch_bounds__(256) void k_fill(uint16_t* __restrict__ out, int64_t n) {
    const int64_t whole = n / kPer, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t i = first; i < whole; i += (int64_t)gridDim.x * 256)
        reinterpret_cast<words4*>(out)[i] = words4{};
    if (first < n - whole * kPer) out[whole * kPer + first] = 0;
}
__global__ __launch_bounds__(256) void k_mark(const int32_t* __restrict__ pos, int64_t n,
                                              int64_t rows, int32_t* __restrict__ slot_of) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * 256) {
        const int64_t p = pos[i];
        if (p >= 0 && p < rows) slot_of[p] = (int32_t)i;
    }
}
// The work-groups behind the tokens' zero the rows without a slot, each wave 16 rows at a
// time.
constexpr int kRestRows = 16;
constexpr int64_t kRestGroups = 4096;
template <int kT>
__device__ __forceinline__ void zero_rest(const Args& a, const int32_t* __restrict__ pos) {
    if (blockIdx.y) return;
    const int lane = threadIdx.x & 63, waves = (int)(blockDim.x >> 6);
    const int64_t first = (int64_t)(blockIdx.x - a.groups) * waves + (threadIdx.x >> 6);
    const int64_t step = (int64_t)(gridDim.x - a.groups) * waves * kRestRows;
    for (int64_t r0 = first * kRestRows; r0 < a.rows; r0 += step) {
        const int64_t r = r0 + lane;
        bool empty = false;
        if (lane < kRestRows && r < a.rows) {
            const int64_t i = a.slot_of[r];
            empty = i < 0 || i >= a.slots || pos[i] != r;
        }
        for (uint64_t left = __ballot(empty); left; left &= left - 1) {
            void* row = row_at<kT>(a.out, (r0 + __builtin_ctzll(left)) * a.H);
            for (int64_t c = lane * kPer; c < a.H; c += 64 * kPer)
                store<kT>(row, c, a.H - c, Raw<kT>{});
        }
    }
}

// Which token and which eight channels a thread has.  kLanes threads to a token (8, 16,
// 32), 256 / kLanes tokens to a work-group; 0: work-group (x, y) has channels
// 8 * blockDim.x * y .. of token x.
template <int kLanes, int kCut>
struct Place {
    int64_t t;
    Piece p;
    __device__ __forceinline__ explicit Place(const Args& a) {
        int c;
        if (kLanes) {
            constexpr int kL = kLanes ? kLanes : 1;
            t = (int64_t)blockIdx.x * (256 / kL) + threadIdx.x / kL;
            c = threadIdx.x % kL;
        } else {
            t = blockIdx.x;
            c = blockIdx.y * blockDim.x + threadIdx.x;
        }
        p = piece<kCut>(c * kPer, (int)a.H);
        if (t >= a.T) p.n = 0;
    }
};
// Packed row of slot s, or -1.
__device__ __forceinline__ int64_t slot_row(const int32_t* pos, int64_t at, int64_t rows) {
    const int64_t p = pos[at];
    return p >= 0 && p < rows ? p : -1;
}

constexpr int kBatch = 8;                    // slots whose rows are asked for together

// Copies know no type: an fp32 row goes as twice as many 16-bit channels, 16 bytes a lane
// next to one another (eight fp32 channels a lane, 4096 x 2048, top 8: 122 us against 54).
template <int kOnce, int kLanes, int kCut>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_sort(Args a,
                                                              const int32_t* __restrict__ pos) {
    constexpr int kT = 1;
    if (blockIdx.x >= a.groups) return zero_rest<kT>(a, pos);
    const Place<kLanes, kCut> at(a);
    if (at.p.n <= 0) return;
    const Raw<kT> r = load<kT, kCut != kTiny>(row_at<kT>(a.a, at.t * a.ld), at.p.at, at.p.n);
    for (int s = 0; s < a.topk; ++s) {
        const int64_t p = slot_row(pos, at.t * a.topk + s, a.rows);
        if (p >= 0)
            store<kT, kCut != kTiny, (kOnce & 2) && kCut == kEven>(row_at<kT>(a.out, p * a.H),
                                                                   at.p.at, at.p.n, r);
    }
}

template <int kY, int kOut, int kOnce, int kLanes, int kCut>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_unsort(Args a,
                                                                const int32_t* __restrict__ pos,
                                                                const float* __restrict__ w) {
    const Place<kLanes, kCut> at(a);
    if (at.p.n <= 0) return;
    float acc[kPer] = {};
    for (int s0 = 0; s0 < a.topk; s0 += kBatch) {
        Raw<kY> r[kBatch];
        float by[kBatch];
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
            const int64_t slot = at.t * a.topk + s0 + s;
            const int64_t p = s0 + s < a.topk ? slot_row(pos, slot, a.rows) : -1;
            r[s] = Raw<kY>{};
            by[s] = 0.0f;
            if (p >= 0) {
                r[s] = load<kY, kCut != kTiny, (kOnce & 1) != 0>(row_at<kY>(a.a, p * a.ld),
                                                                 at.p.at, at.p.n);
                by[s] = w ? w[slot] : 1.0f;
            }
        }
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
            if (s0 + s >= a.topk) break;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = fmaf(by[s], r[s].get(i), acc[i]);
        }
    }
    store<kOut, kCut != kTiny>(row_at<kOut>(a.out, at.t * a.ld), at.p.at, at.p.n, pack<kOut>(acc));
}

// kLanes 0: a work-group per token and `per` slots, its threads over the row, again where it
// is longer.  dy may be y: a thread has loaded its channels of a slot's row when it stores
// them, but another wave, or a later turn over the row, may have the last, partial eight,
// and must then leave alone the channels that it shares with the eight before.
template <int kG, int kY, int kOnce, int kLanes, int kCut>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_unsort_grad(
    Args a, const int32_t* __restrict__ pos, const float* __restrict__ w) {
    constexpr int kMaxWaves = kLanes ? 1 : 16, kL = kLanes ? kLanes : 64;
    __shared__ float s_dot[kLanes ? 1 : kMaxTopk][kMaxWaves];
    if (blockIdx.x >= a.groups) return zero_rest<kY>(a, pos);
    const Place<kLanes, kCut> at(a);
    const int from = kLanes ? 0 : blockIdx.y * a.per;
    const int end = kLanes || from + a.per > a.topk ? a.topk : from + a.per;
    const int step = kLanes ? 1 : (int)blockDim.x * kPer;
    int c = kLanes ? 0 : (int)threadIdx.x * kPer;
    for (int first = 1;; first = 0) {
        const Piece p = kLanes ? at.p : piece<kCut>(c, (int)a.H);
        Raw<kG> g = {};
        if (p.n > 0) g = load<kG, kCut != kTiny>(row_at<kG>(a.a, at.t * a.H), p.at, p.n);
        for (int s0 = from; s0 < end; s0 += kBatch) {
            Raw<kY> y[kBatch];
            int64_t row[kBatch];
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int64_t slot = at.t * a.topk + s0 + s;
                row[s] = s0 + s < end && (!kLanes || at.t < a.T) ? slot_row(pos, slot, a.rows)
                                                                    : -1;
                y[s] = Raw<kY>{};
                if (a.dw && row[s] >= 0 && p.n > 0)
                    y[s] = load<kY, kCut != kTiny, (kOnce & 1) != 0>(
                        row_at<kY>(a.y, row[s] * a.H), p.at, p.n);
            }
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                if (s0 + s >= end) break;
                const int64_t slot = at.t * a.topk + s0 + s;
                if (a.out && row[s] >= 0 && p.n > 0) {
                    const float by = w ? w[slot] : 1.0f;
                    float d[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i) d[i] = by * g.get(i);
                    void* out = row_at<kY>(a.out, row[s] * a.H);
                    if (kCut == kOdd && p.from > 0 && a.out == a.y)
                        store_own<kY>(out, p, pack<kY>(d));
                    else
                        store<kY, kCut != kTiny, (kOnce & 2) && kCut == kEven>(out, p.at, p.n,
                                                                               pack<kY>(d));
                }
                if (a.dw) {
                    float dot = 0.0f;
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (kCut != kOdd || i >= p.from) dot = fmaf(g.get(i), y[s].get(i), dot);
                    dot = lanes_sum<kL>(row[s] >= 0 ? dot : 0.0f);   // g may not be finite
                    if (kLanes) {
                        if (threadIdx.x % kL == 0 && at.t < a.T) a.dw[slot] = dot;
                    } else if ((threadIdx.x & 63) == 0) {
                        float& all = s_dot[kLanes ? 0 : s0 + s][kLanes ? 0 : threadIdx.x >> 6];
                        all = first ? dot : all + dot;
                    }
                }
            }
        }
        if (kLanes) return;
        c += step;
        if (c - (int)threadIdx.x * kPer >= a.H) break;
    }
    if (kLanes || !a.dw) return;
    __syncthreads();
    for (int s = from + threadIdx.x; s < end; s += blockDim.x) {
        float v = s_dot[kLanes ? 0 : s][0];
        for (int i = 1; i < (int)(blockDim.x >> 6); ++i) v += s_dot[kLanes ? 0 : s][kLanes ? 0 : i];
        a.dw[at.t * a.topk + s] = v;
    }
}

// ------------------------------------------------------------------- host --
// Packed rows beyond what the caches keep go past them (kOnce: 1 their loads, 2 their
// stores), us: loads from 16 MB on (gradient 4096 x 2048, top 8, bf16 53 against 63, unsort
// 28 / 30; 16384 x 128, top 2, 7.9 / 7.0), stores from 192 MB on (sort 16384 x 4096, top 8,
// bf16 212 / 242; 4096 x 2048 27.4 / 28.0, but with the call that reads them 55 / 48.7).
// Stores only of whole 16 bytes, neither of fp32, whose 32 bytes of a lane are two accesses
// to a line (the gradient 16384 x 4096, top 4, fp32 511 / 469).
constexpr int64_t kOnceLoads = (int64_t)16 << 20, kOnceStores = (int64_t)192 << 20;

struct Shape {
    int lanes, threads;
    dim3 grid;
};
// `parts`: a row may be several work-groups' (512 threads; 128 where there are few rows:
// sort 64 x 4096, top 8, fp32 4.5 us against 5.5).
inline Shape shape_of(int64_t T, int64_t H, bool parts) {
    const int64_t chunks = (H + kPer - 1) / kPer;
    for (int l = 8; l <= 32; l *= 2)
        if (chunks <= l) return {l, 256, dim3((unsigned)((T * l + 255) / 256))};
    int threads = (int)(chunks < 1024 ? (chunks + 63) / 64 * 64 : 1024);
    if (!parts) return {0, threads, dim3((unsigned)T)};
    const int most = T * ((chunks + 511) / 512) < 512 ? 128 : 512;
    if (threads > most) threads = most;
    return {0, threads, dim3((unsigned)T, (unsigned)((chunks + threads - 1) / threads))};
}

// A launch has fewer than 2^32 threads: tokens of one launch, at most.
constexpr int64_t kLaunchTokens = (int64_t)1 << 21;

template <int kValue>
using Int = std::integral_constant<int, kValue>;
// f(kOnce, kLanes, kCut) of rows of H channels; kOnce for work-groups of one token only.
template <int kOnce, typename F>
void with_shape(const Shape& p, int64_t H, F f) {
    const Cut cut = cut_of(H);
    if (cut == kTiny) f(Int<0>{}, Int<8>{}, Int<kTiny>{});
    else if (p.lanes == 8 && cut == kEven) f(Int<0>{}, Int<8>{}, Int<kEven>{});
    else if (p.lanes == 8) f(Int<0>{}, Int<8>{}, Int<kOdd>{});
    else if (p.lanes == 16 && cut == kEven) f(Int<0>{}, Int<16>{}, Int<kEven>{});
    else if (p.lanes == 16) f(Int<0>{}, Int<16>{}, Int<kOdd>{});
    else if (p.lanes == 32 && cut == kEven) f(Int<0>{}, Int<32>{}, Int<kEven>{});
    else if (p.lanes == 32) f(Int<0>{}, Int<32>{}, Int<kOdd>{});
    else if (cut == kEven) f(Int<kOnce>{}, Int<0>{}, Int<kEven>{});
    else f(Int<kOnce>{}, Int<0>{}, Int<kOdd>{});
}

// Work-groups for the rows without a slot, behind those with tokens.
inline void add_rest(Args& a, Shape& p) {
    a.groups = p.grid.x;
    if (!a.slot_of) return;
    const int64_t each = p.threads / 64 * kRestRows, n = (a.rows + each - 1) / each;
    p.grid.x += (unsigned)(n < kRestGroups ? n : kRestGroups);
}
// What comes before them: the whole output zeroed, or the inverse written (`bytes`: of the
// output's rows).
inline int before_rest(void* out, int64_t bytes, const int32_t* pos, int64_t slots, int64_t rows,
                       void* ws, hipStream_t s) {
    const bool fill = bytes <= kFillBytes;
    const int64_t n = fill ? bytes / 2 : slots, each = fill ? 256 * kPer : 256;
    const int64_t groups = (n + each - 1) / each;
    const dim3 grid((unsigned)(groups < 4096 ? groups : 4096));
    if (fill)
        hipLaunchKernelGGL(k_fill, grid, dim3(256), 0, s, (uint16_t*)out, n);
    else if (slots)
        hipLaunchKernelGGL(k_mark, grid, dim3(256), 0, s, pos, slots, rows, (int32_t*)ws);
    QUADS_CHECK_LAUNCH();
    return QUADS_OK;
}

// `bytes`: of the packed rows that the slots name.
inline void launch_sort(Args& a, const int32_t* pos, int64_t bytes, hipStream_t s) {
    Shape p = shape_of(a.T, a.H, true);
    add_rest(a, p);
    auto go = [&](auto once, auto lanes, auto cut) {
        hipLaunchKernelGGL((k_sort<once(), lanes(), cut()>), p.grid, dim3(p.threads), 0, s, a, pos);
    };
    if (bytes > kOnceStores) with_shape<2>(p, a.H, go);
    else with_shape<0>(p, a.H, go);
}
template <int kY, int kOut>
void launch_unsort(const Args& a, const int32_t* pos, const float* w, int64_t bytes,
                   hipStream_t s) {
    const Shape p = shape_of(a.T, a.H, true);
    auto go = [&](auto once, auto lanes, auto cut) {
        hipLaunchKernelGGL((k_unsort<kY, kOut, once(), lanes(), cut()>), p.grid, dim3(p.threads), 0,
                           s, a, pos, w);
    };
    if constexpr (kY != 0) {
        if (bytes > kOnceLoads) return with_shape<1>(p, a.H, go);
    }
    with_shape<0>(p, a.H, go);
}
// Slots of a work-group: all of them, fewer where there are few tokens (64 x 2048, top 8,
// bf16: 6.7 us against 4.2; 64 x 4096 fp32 8.7 / 6.7).
inline int slots_of(int64_t T, int topk) {
    const int64_t per = T * topk / 512;
    return per < 1 ? 1 : (per < topk ? (int)per : topk);
}
template <int kG, int kY>
void launch_grad(Args& a, const int32_t* pos, const float* w, int64_t bytes, hipStream_t s) {
    Shape p = shape_of(a.T, a.H, false);
    if (!p.lanes) p.grid.y = (a.topk + a.per - 1) / a.per;
    add_rest(a, p);
    auto go = [&](auto once, auto lanes, auto cut) {
        hipLaunchKernelGGL((k_unsort_grad<kG, kY, once(), lanes(), cut()>), p.grid, dim3(p.threads),
                           0, s, a, pos, w);
    };
    if constexpr (kY != 0) {
        if (bytes > kOnceStores) return with_shape<3>(p, a.H, go);
        if (bytes > kOnceLoads) return with_shape<1>(p, a.H, go);
    }
    with_shape<0>(p, a.H, go);
}

inline int check(int64_t T, int64_t H, int64_t ld, int32_t topk, int64_t rows) {
    if (T < 0 || T >= ((int64_t)1 << 24) || H < 1 || H >= kMaxH || ld < H || ld >= kMaxStride)
        return QUADS_ESHAPE;
    if (topk < 1 || topk > kMaxTopk || rows < 0 || rows >= ((int64_t)1 << 31) ||
        T * topk >= ((int64_t)1 << 31))
        return QUADS_ESHAPE;
    return QUADS_OK;
}

// The way back, in launches of at most kLaunchTokens tokens and kPartChannels channels.
constexpr int64_t kPartChannels = (int64_t)1 << 24;
inline int back(const void* y, int y_dtype, int64_t rows, const int32_t* pos, const float* topk_w,
                int64_t T, int32_t topk, int64_t H, void* out, int out_dtype, hipStream_t s) {
    const bool yb = y_dtype == QUADS_OUT_BF16, ob = out_dtype == QUADS_OUT_BF16;
    const int64_t bytes = T * topk * H * (yb ? 2 : 4);
    for (int64_t t = 0; t < T; t += kLaunchTokens) {
        for (int64_t c = 0; c < H; c += kPartChannels) {
            Args a = {};
            a.a = (const char*)y + c * (yb ? 2 : 4);
            a.out = (char*)out + (t * H + c) * (ob ? 2 : 4);
            a.T = T - t < kLaunchTokens ? T - t : kLaunchTokens;
            a.H = H - c < kPartChannels ? H - c : kPartChannels;
            a.ld = H;
            a.rows = rows;
            a.topk = topk;
            const int32_t* p = pos + t * topk;
            const float* w = topk_w ? topk_w + t * topk : nullptr;
            if (yb && ob) launch_unsort<1, 1>(a, p, w, bytes, s);
            else if (yb) launch_unsort<1, 0>(a, p, w, bytes, s);
            else if (ob) launch_unsort<0, 1>(a, p, w, bytes, s);
            else launch_unsort<0, 0>(a, p, w, bytes, s);
            QUADS_CHECK_LAUNCH();
        }
    }
    return QUADS_OK;
}

}  // namespace sorting
}  // namespace quads

using namespace quads;

extern "C" size_t quads_moe_sort_ws(int64_t rows, int64_t H, int dtype, int zero_rest) {
    if (!zero_rest || rows <= 0 || rows >= ((int64_t)1 << 31) || H < 1 || H >= block::kMaxH)
        return 0;
    const int64_t bytes = rows * H * (dtype == QUADS_OUT_BF16 ? 2 : 4);
    return bytes <= sorting::kFillBytes ? 0 : align_up((size_t)rows * 4, 256);
}

extern "C" int quads_moe_sort(const void* x, int dtype, int64_t T, int64_t H, int64_t ldx,
                              const int32_t* pos, int32_t topk, int64_t rows, int zero_rest,
                              void* out, void* ws, size_t ws_bytes, void* stream) {
    using namespace sorting;
    if (int e = check(T, H, ldx, topk, rows)) return e;
    if (!ok_type(dtype) || (zero_rest != 0 && zero_rest != 1)) return QUADS_EINVAL;
    if (rows == 0 || (T == 0 && !zero_rest)) return QUADS_OK;
    if (!ok_ptr(out) || (T > 0 && (!ok_ptr(x) || !ok_ptr4(pos) || x == out))) return QUADS_EINVAL;
    const size_t need = quads_moe_sort_ws(rows, H, dtype, zero_rest);
    if (need && (ws_bytes < need || !ok_ptr(ws))) return QUADS_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    const int size = dtype == QUADS_OUT_BF16 ? 2 : 4;
    const int64_t slots = T * topk, bytes = slots * H * size;
    if (zero_rest)
        if (int e = before_rest(out, rows * H * size, pos, slots, rows, ws, s)) return e;
    if (T == 0 && !need) return QUADS_OK;
    for (int64_t t = 0; t < T || t == 0; t += kLaunchTokens) {
        Args a = {};
        a.a = (const char*)x + t * ldx * size;
        a.out = out;
        a.T = T - t < kLaunchTokens ? T - t : kLaunchTokens;
        a.H = H * size / 2;
        a.ld = ldx * size / 2;
        a.rows = rows;
        a.topk = topk;
        a.slot_of = need && t == 0 ? (const int32_t*)ws : nullptr;
        a.slots = slots;
        launch_sort(a, pos + t * topk, bytes, s);
        QUADS_CHECK_LAUNCH();
    }
    return QUADS_OK;
}

extern "C" int quads_moe_unsort(const void* y, int y_dtype, int64_t rows, const int32_t* pos,
                                const float* topk_w, int64_t T, int32_t topk, int64_t H, void* out,
                                int out_dtype, void* stream) {
    using namespace sorting;
    if (int e = check(T, H, H, topk, rows)) return e;
    if (!ok_type(y_dtype) || !ok_type(out_dtype)) return QUADS_EINVAL;
    if (T == 0) return QUADS_OK;
    if ((rows > 0 && !ok_ptr(y)) || !ok_ptr4(pos) || !ok_opt4(topk_w) || !ok_ptr(out) || y == out)
        return QUADS_EINVAL;
    return sorting::back(y, y_dtype, rows, pos, topk_w, T, topk, H, out, out_dtype,
                         (hipStream_t)stream);
}

// Any number of slots, tokens and rows' eights; pos names T * topk rows.
extern "C" int quads_moe_combine(const void* y, int y_dtype, const int32_t* pos,
                                 const float* topk_w, int64_t T, int32_t topk, int64_t N,
                                 float* out, void* stream) {
    if (y_dtype != QUADS_OUT_F32 && y_dtype != QUADS_OUT_BF16) return QUADS_EINVAL;
    if (T < 0 || topk < 1 || N <= 0 || N % 8) return QUADS_ESHAPE;
    if (T > 0 && (!ok_ptr(y) || !ok_ptr(pos) || !ok_ptr(topk_w) || !ok_ptr(out)))
        return QUADS_EINVAL;
    return sorting::back(y, y_dtype, T * topk, pos, topk_w, T, topk, N, out, QUADS_OUT_F32,
                         (hipStream_t)stream);
}

extern "C" int quads_moe_unsort_backward(const void* g, int g_dtype, const void* y, int y_dtype,
                                         int64_t rows, const int32_t* pos, const float* topk_w,
                                         int64_t T, int32_t topk, int64_t H, int zero_rest,
                                         void* dy, float* dw, void* ws, size_t ws_bytes,
                                         void* stream) {
    using namespace sorting;
    if (int e = check(T, H, H, topk, rows)) return e;
    if (!ok_type(g_dtype) || !ok_type(y_dtype) || (zero_rest != 0 && zero_rest != 1))
        return QUADS_EINVAL;
    if (dw && !topk_w) return QUADS_EINVAL;
    const bool rest = zero_rest && dy && rows > 0;
    if ((!dy && !dw) || (T == 0 && !rest)) return QUADS_OK;
    if (!ok_opt_ptr(dy) || !ok_opt4(dw) ||
        (T > 0 && (!ok_ptr(g) || (rows > 0 && dw && !ok_ptr(y)) || !ok_ptr4(pos) ||
                   !ok_opt4(topk_w) || dy == g)))
        return QUADS_EINVAL;
    if (rest && dy == y) return QUADS_EINVAL;
    const size_t need = quads_moe_sort_ws(rows, H, y_dtype, rest);
    if (need && (ws_bytes < need || !ok_ptr(ws))) return QUADS_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    const bool gb = g_dtype == QUADS_OUT_BF16, yb = y_dtype == QUADS_OUT_BF16;
    const int64_t slots = T * topk, bytes = slots * H * (yb ? 2 : 4);
    if (rest)
        if (int e = before_rest(dy, rows * H * (yb ? 2 : 4), pos, slots, rows, ws, s)) return e;
    if (T == 0 && !need) return QUADS_OK;
    for (int64_t t = 0; t < T || t == 0; t += kLaunchTokens) {
        Args a = {};
        a.a = (const char*)g + t * H * (gb ? 2 : 4);
        a.y = y;
        a.out = dy;
        a.dw = dw ? dw + t * topk : nullptr;
        a.T = T - t < kLaunchTokens ? T - t : kLaunchTokens;
        a.H = H;
        a.rows = rows;
        a.topk = topk;
        a.per = slots_of(T, topk);
        a.slot_of = need && t == 0 ? (const int32_t*)ws : nullptr;
        a.slots = slots;
        const int32_t* p = pos + t * topk;
        const float* w = topk_w ? topk_w + t * topk : nullptr;
        if (gb && yb) launch_grad<1, 1>(a, p, w, bytes, s);
        else if (gb) launch_grad<1, 0>(a, p, w, bytes, s);
        else if (yb) launch_grad<0, 1>(a, p, w, bytes, s);
        else launch_grad<0, 0>(a, p, w, bytes, s);
        QUADS_CHECK_LAUNCH();
    }
    return QUADS_OK;
}
