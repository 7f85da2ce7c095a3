// Norms of queries and keys, head by head, with the position rotation in the same pass:
//
//   y = x (mean(x^2) + eps)^-1/2 w   for each row x of `dim` values (y = x without a weight w), then
//   (y_u cos t - y_v sin t, y_v cos t + y_u sin t)   for each pair (u, v) of the first `rotated` values,
//
// t = position * inv_freq of the pair.  The result is rounded to x's type, or quantised to E4M3 with a
// scale a row as cache_write does.
//
// Bound by the bytes where the instructions allow it: each value is read and written once, but a row of 128
// takes some 60 warp instructions for two.  A row goes to dim / 8 lanes, each with two runs of four values
// that lie `rotated / 2` apart (side by side for interleaved pairs and past the rotated values), so both
// values of a pair are in one lane and nothing but the sum of squares (and the largest magnitude) crosses
// lanes.  Such a group of lanes takes up to 10 heads (of 16 bits) of one tensor and token, which all come into
// shared memory at once, and keeps the sines' and cosines' products with the weights in registers; a block's
// tokens share a table of sines and cosines, made by all of its threads while the rows are on their way.
//
// Measured: 16384 tokens x 40 heads of 128 in bfloat16 (336 MB) 53.0 us, 6.3 TB/s of 6.8; with rows loaded straight
// into registers 82, heads of both tensors in one group 64.  8192 tokens x 32 heads to E4M3 (102 MB) 24.2 us, where
// the instructions decide (74 % of the issue slots); twice as many values a lane, with a third fewer instructions, took
// 25.6 for 25.1, since the registers leave fewer warps.
#pragma once

#include <type_traits>

#include "paged_common.cuh"
#include "sm103_ptx.cuh"

namespace fp8mqa {

constexpr int kRotateThreads = 128;

// Heads of a group of lanes, at most, and the shared memory for `rows` of each: eight blocks of an SM have room for
// 10 of 16 bits (16 take 59 us where 10 take 53, 4 take 63).
template <class X>
constexpr int kRotateHeads = 20 / int(sizeof(X));
template <class X>
constexpr int rotate_smem(int rows) { return kRotateThreads * 8 * int(sizeof(X)) * rows; }

// To E4M3 the norm's factor, eps^-1/2 at most, goes into the one that quantises, 448 / kTinyMax = 4.48e32 at most (of a
// row of zeros, say).  From this eps on the product is under 3.2e38; below, kernels of their own look whether it is finite
// (the 8192 x 32 rows above take 25.7 us with that look, 24.3 without).
constexpr float kRotateEps = 2e-12f;

struct NormRotateParams {
    const void* x[2];
    int64_t row_stride[2], head_stride[2];  // elements
    const void* weight[2];
    int32_t weight_f32[2];
    void* out[2];
    int64_t out_row_stride[2], out_head_stride[2];
    float* out_scale[2];  // [T, heads], for E4M3
    int32_t heads[2];
    int32_t units[2];     // groups of lanes that a token's heads of each tensor go to,
    int32_t per_unit;     // so many each
    FastDiv by_units;     // all of a token
    int32_t T;
    const void* positions;
    int32_t wide_positions;  // 64 bits
    const float* inv_freq;
    int32_t rotated;
    float eps;
    PagedBounds bounds;
};

// f radians as a 64-bit fraction of a turn, f = m 2^e / 2 pi with the 24 bits m of f's mantissa: m times
// round(2^66 / 2 pi), shifted into place, correct to one in its last place or 2^-64 of itself.
__device__ __forceinline__ uint64_t turn_of(float f)
{
    constexpr uint64_t kTurn = 0xA2F9836E4E44152AULL;
    const uint32_t bits = __float_as_uint(f);
    const int e = int(bits >> 23 & 0xFFu);
    const uint32_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const uint64_t lo = m * (kTurn & 0xFFFFFFFFu), mid = m * (kTurn >> 32) + (lo >> 32);
    // the product, 88 bits, is mid 2^32 + (lo mod 2^32), in units of 2^-s of a place
    const int s = 152 - max(e, 1);
    uint64_t turn;
    if (s >= 32) turn = s < 96 ? mid >> (s - 32) : 0;
    else if (s >= 0) turn = (mid << (32 - s)) | (uint32_t(lo) >> s);
    else turn = s > -64 ? ((mid << 32) | uint32_t(lo)) << -s : 0;
    return bits >> 31 ? 0 - turn : turn;
}

// A lane's eight values of a row, two runs of four.
template <class X>
struct alignas(16) Eight {
    X v[8];
};

// From shared memory, or (kVec: on 16 bytes) from the weights.  kAside: the second run follows the first.
template <class X, bool kVec, bool kAside>
__device__ __forceinline__ Eight<X> load8(const X* a, const X* b)
{
    Eight<X> r;
    uint4* const q = reinterpret_cast<uint4*>(&r);
    if constexpr (!kVec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = j < 4 ? a[j] : b[j - 4];
    } else if constexpr (sizeof(X) == 4) {
        q[0] = *reinterpret_cast<const uint4*>(a);
        q[1] = *reinterpret_cast<const uint4*>(b);
    } else if constexpr (kAside) {
        q[0] = *reinterpret_cast<const uint4*>(a);
    } else {
        const uint2 lo = *reinterpret_cast<const uint2*>(a), hi = *reinterpret_cast<const uint2*>(b);
        q[0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    return r;
}

template <class X>
__device__ __forceinline__ Eight<X> eight_of(const float* y)
{
    Eight<X> r;
    if constexpr (sizeof(X) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = y[j];
    } else {
        constexpr bool kBf16 = std::is_same_v<X, __nv_bfloat16>;
        *reinterpret_cast<uint4*>(&r) = make_uint4(pack16<kBf16>(y[0], y[1]), pack16<kBf16>(y[2], y[3]),
                                                   pack16<kBf16>(y[4], y[5]), pack16<kBf16>(y[6], y[7]));
    }
    return r;
}

template <class X, bool kVec, bool kAside>
__device__ __forceinline__ void store8(const PagedBounds& bounds, int kind, X* a, X* b, const Eight<X>& r)
{
    if (!in_bounds(bounds, kind, a, 4 * sizeof(X)) || !in_bounds(bounds, kind, b, 4 * sizeof(X))) return;
    const uint4* const q = reinterpret_cast<const uint4*>(&r);
    if constexpr (!kVec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) (j < 4 ? a[j] : b[j - 4]) = r.v[j];
    } else if constexpr (sizeof(X) == 4) {
        *reinterpret_cast<uint4*>(a) = q[0];
        *reinterpret_cast<uint4*>(b) = q[1];
    } else if constexpr (kAside) {
        *reinterpret_cast<uint4*>(a) = q[0];
    } else {
        *reinterpret_cast<uint2*>(a) = make_uint2(q[0].x, q[0].y);
        *reinterpret_cast<uint2*>(b) = make_uint2(q[0].z, q[0].w);
    }
}

// X: x's type.  kE4m3: the result is E4M3 with scales, else of x's type.  kVec: x, its weights and the result lie on
// 16 bytes (E4M3: on 8).  kInterleaved: how values pair, side by side or apart.  kSmallEps: for E4M3 with an eps under
// kRotateEps.
template <class X, int kDim, bool kE4m3, bool kVec, bool kInterleaved, bool kSmallEps>
__global__ void __launch_bounds__(kRotateThreads, 8) norm_rotate_kernel(const __grid_constant__ NormRotateParams p)
{
    constexpr int kLanes = kDim / 8, kGroups = kRotateThreads / kLanes;
    constexpr int kRows = 2;  // worked on at once
    extern __shared__ __align__(16) uint8_t s_rows[];  // [group][row][kDim]
    __shared__ float2 s_turns[kGroups][kDim / 2];      // sine and cosine of the block's tokens
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int64_t unit0 = int64_t(blockIdx.x) * kGroups;  // the block's first (under 2^31)
    const int units = p.units[0] + p.units[1];
    const int64_t unit = unit0 + group;
    const bool there = unit < int64_t(p.T) * units;
    const int32_t t0 = p.by_units.of(int32_t(unit0));     // its token
    const int32_t t = there ? p.by_units.of(int32_t(unit)) : t0;
    const int part = int(unit - int64_t(t) * units);      // of the token's units
    const int which = there && part >= p.units[0];
    const int h0 = (which ? part - p.units[0] : part) * p.per_unit;
    const int n = there ? min(p.per_unit, p.heads[which] - h0) : 0;  // heads

    // ---- the lane's two runs of four values; for pairs (i, i + rotated / 2) they are as far apart
    const bool turns = 8 * lane < p.rotated;
    const bool apart = !kInterleaved && turns;
    const int at_a = apart ? 4 * lane : 8 * lane, at_b = apart ? p.rotated / 2 + 4 * lane : 8 * lane + 4;
    using Out = std::conditional_t<kE4m3, uint8_t, X>;
    X* const s_mine = reinterpret_cast<X*>(s_rows) + group * p.per_unit * kDim;

    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the heads come into shared memory, a lane's eight values of each next to those of the lane before
    {
        const int64_t step = p.head_stride[which];
        const X* from = static_cast<const X*>(p.x[which]) + t * p.row_stride[which] + h0 * step + 8 * lane;
        X* to = s_mine + 8 * lane;
        for (int i = 0; i < n; ++i, from += step, to += kDim) {
            const bool ok = in_bounds(p.bounds, kMemRows + which, from, 8 * sizeof(X));
            if constexpr (kVec) {
#pragma unroll
                for (int j = 0; j < 8; j += 16 / sizeof(X)) copy16(ptx::smem_addr(to + j), from + j, ok);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) to[j] = ok ? from[j] : from_float<X>(0.0f);
            }
        }
        copy_commit();
    }

    // ---- the block's tokens' sines and cosines
    constexpr int kPairs = kDim / 2;
    const int pair = threadIdx.x % kPairs;
    const int64_t unit_end = min(unit0 + kGroups, int64_t(p.T) * units);
    const int64_t t_end = p.by_units.of(int32_t(unit_end - 1)) + int64_t(1);
    for (int token = threadIdx.x / kPairs; t0 + token < t_end && 2 * pair < p.rotated; token += kRotateThreads / kPairs) {
        int64_t pos = 0;
        if (p.wide_positions) {
            const int64_t* const at = static_cast<const int64_t*>(p.positions) + t0 + token;
            if (in_bounds(p.bounds, kMemPositions, at, 8)) pos = *at;
        } else {
            const int32_t* const at = static_cast<const int32_t*>(p.positions) + t0 + token;
            if (in_bounds(p.bounds, kMemPositions, at, 4)) pos = *at;
        }
        const float* const at = p.inv_freq + pair;
        const float f = in_bounds(p.bounds, kMemFreq, at, 4) ? *at : 0.0f;
        // in halves of a turn, [-1, 1)
        const float half = float(int32_t((turn_of(f) * uint64_t(pos)) >> 32)) * 0x1p-31f;
        float2 sc;
        sincospif(half + (f - f), &sc.x, &sc.y);  // (f - f: NaN of a frequency that is not finite)
        s_turns[token][pair] = sc;
    }
    __syncthreads();

    copy_wait<0>();
    __syncwarp();

    // ---- the pairs' factors: out_u = u cu - v sv, out_v = v cv + u su, with the weights in them.  Pair j is value
    // j of either run, or values 2 j and 2 j + 1 of the two runs
    float cu[4], su[4], cv[4], sv[4];
    const bool norm = p.weight[which] != nullptr;
    {
        float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (norm) {
            const auto values = [&](auto* from) {
                if (in_bounds(p.bounds, kMemWeight + which, from, kDim * sizeof(*from))) {
                    using W = std::remove_cv_t<std::remove_pointer_t<decltype(from)>>;
                    const Eight<W> e = load8<W, kVec, kInterleaved>(from + at_a, from + at_b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = to_float(e.v[j]);
                }
            };
            if (p.weight_f32[which]) values(static_cast<const float*>(p.weight[which]));
            else values(static_cast<const X*>(p.weight[which]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float wu = w[kInterleaved ? 2 * j : j], wv = w[kInterleaved ? 2 * j + 1 : 4 + j];
            const float2 sc = turns ? s_turns[t - t0][4 * lane + j] : make_float2(0.0f, 1.0f);
            cu[j] = wu * sc.y;
            su[j] = wu * sc.x;
            cv[j] = wv * sc.y;
            sv[j] = wv * sc.x;
        }
    }

    // ---- the heads, all lanes of a warp together (they exchange sums): a group past its last one does nothing
    const int64_t out_step = p.out_head_stride[which];
    Out* out = static_cast<Out*>(p.out[which]) + t * p.out_row_stride[which] + h0 * out_step;
    float* out_scale = kE4m3 ? p.out_scale[which] + int64_t(t) * p.heads[which] + h0 : nullptr;
    const X* row = s_mine;
    for (int i = 0; i < p.per_unit; i += kRows, row += kRows * kDim) {
        float y[kRows][8], by[kRows], top[kRows];  // y: as it lies in the runs
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const X* const from = i + r < n ? row + r * kDim : row;
            const Eight<X> raw = load8<X, true, kInterleaved>(from + at_a, from + at_b);
            by[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[r][j] = to_float(raw.v[j]);
                by[r] = fmaf(y[r][j], y[r][j], by[r]);
            }
        }
        // (without a weight too: a warp's groups may be of both tensors, and all its lanes exchange)
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2)
#pragma unroll
            for (int r = 0; r < kRows; ++r) by[r] += __shfl_xor_sync(~0u, by[r], o);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            by[r] = norm ? rsqrtf(fmaf(by[r], 1.0f / kDim, p.eps)) : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float &u = y[r][kInterleaved ? 2 * j : j], &v = y[r][kInterleaved ? 2 * j + 1 : 4 + j];
                float nu = u * cu[j], nv = v * cv[j];
                if (turns) {  // (others have nothing to do with one another: one may be infinite)
                    nu = fmaf(-v, sv[j], nu);
                    nv = fmaf(u, su[j], nv);
                }
                u = kE4m3 ? nu : nu * by[r];
                v = kE4m3 ? nv : nv * by[r];
            }
        }
        if constexpr (kE4m3) {  // (the row's factor joins the scale's)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                top[r] = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; j += 2) top[r] = max_nan(top[r], fabsf(y[r][j]), fabsf(y[r][j + 1]));
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o /= 2)
#pragma unroll
                for (int r = 0; r < kRows; ++r) top[r] = max_nan(top[r], __shfl_xor_sync(~0u, top[r], o));
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (i + r >= n) break;
            const int kind = which ? kMemOut2 : kMemOut;
            if constexpr (kE4m3) {
                const float a = max_nan(top[r] * by[r], kTinyMax), to_codes = __fdiv_rn(kE4m3Max, a);
                float inv = by[r] * to_codes;
                if constexpr (kSmallEps) {
                    if (!(inv <= 3.402823466e38f)) {  // one after the other
                        inv = to_codes;
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[r][j] *= by[r];
                    }
                }
                uint32_t four[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float* const z = y[r] + 4 * j;
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                        make_float2(__fmul_rn(z[0], inv), __fmul_rn(z[1], inv)), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(__fmul_rn(z[2], inv), __fmul_rn(z[3], inv)), __NV_SATFINITE, __NV_E4M3);
                    four[j] = lo | hi << 16;
                }
                if constexpr (kVec && kInterleaved) {
                    if (in_bounds(p.bounds, kind, out + at_a, 8))
                        *reinterpret_cast<uint2*>(out + at_a) = make_uint2(four[0], four[1]);
                } else {
                    if (in_bounds(p.bounds, kind, out + at_a, 4)) *reinterpret_cast<uint32_t*>(out + at_a) = four[0];
                    if (in_bounds(p.bounds, kind, out + at_b, 4)) *reinterpret_cast<uint32_t*>(out + at_b) = four[1];
                }
                if (lane == 0 && in_bounds(p.bounds, which ? kMemOutScale2 : kMemOutScale, out_scale, 4))
                    *out_scale = __fmul_rn(a, 1.0f / kE4m3Max);
                ++out_scale;
            } else {
                store8<X, kVec, kInterleaved>(p.bounds, kind, out + at_a, out + at_b, eight_of<X>(y[r]));
            }
            out += out_step;
        }
    }
}
}  // namespace fp8mqa
