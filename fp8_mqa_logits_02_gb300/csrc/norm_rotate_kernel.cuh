// Norms of queries and keys, head by head, with the position rotation in the same pass:
//
//   y = x (mean(x^2) + eps)^-1/2 w   for each row x of `dim` values (y = x without a weight w), then
//   (y_a cos t - y_b sin t, y_b cos t + y_a sin t)   for each pair (a, b) of the first `rotated` values,
//
// t = position * inv_freq of the pair.  The result is rounded to x's type, or quantised to E4M3 with a
// scale a row as cache_write does.
//
// Bound by the bytes: each value is read and written once, with some 10 instructions a value between.  A
// row goes to dim / 8 lanes, each with two runs of four values that lie `rotated / 2` apart (side by side
// for interleaved pairs and past the rotated values), so both values of a pair are in one lane and nothing
// but the sum of squares (and the largest magnitude) crosses lanes.  Such a group of lanes takes several
// heads of one token: sine and cosine, and their products with the weights, are made once for them.
//
// Far positions: a product position * inv_freq of 10^5 has no correct digit past the fifth in 32 bits.
// The frequency is taken as a 64-bit fraction of a turn (one fp64 product, correct to 2^-52 of it), so that
// its product with an integer position wraps around by itself; what is left is under half a turn, exact to
// 32 bits of it.
#pragma once

#include "paged_common.cuh"

namespace fp8mqa {

constexpr int kRotateThreads = 256;

struct NormRotateParams {
    const void* x[2];
    int64_t row_stride[2], head_stride[2];  // elements
    const void* weight[2];
    int32_t weight_f32[2];
    void* out[2];
    int64_t out_row_stride[2], out_head_stride[2];
    float* out_scale[2];  // [T, heads], for E4M3
    int32_t heads[2];
    int32_t units[2];     // of a token's heads of each tensor
    int32_t per_unit;     // heads
    FastDiv by_units;     // all units of a token
    int64_t T;
    const void* positions;
    int32_t wide_positions;  // 64 bits
    const float* inv_freq;
    int32_t rotated, interleaved;
    float eps;
    PagedBounds bounds;
};

// Four values side by side, as floats; kVec: they lie on their own size.
template <class X, bool kVec>
__device__ __forceinline__ void load4(const PagedBounds& bounds, int kind, const X* x, float (&v)[4])
{
    alignas(16) X raw[4];
    if (!in_bounds(bounds, kind, x, sizeof(raw))) {
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = from_float<X>(0.0f);
    } else if constexpr (kVec && sizeof(X) == 4) {
        *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(x);
    } else if constexpr (kVec) {
        *reinterpret_cast<uint2*>(raw) = *reinterpret_cast<const uint2*>(x);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = x[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = to_float(raw[j]);
}

template <class X, bool kVec>
__device__ __forceinline__ void store4(const PagedBounds& bounds, int kind, X* to, const float (&v)[4])
{
    if (!in_bounds(bounds, kind, to, 4 * sizeof(X))) return;
    alignas(16) X raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) raw[j] = from_float<X>(v[j]);
    if constexpr (kVec && sizeof(X) == 4) {
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(raw);
    } else if constexpr (kVec) {
        *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(raw);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = raw[j];
    }
}

// X: x's type.  kE4m3: the result is E4M3 with scales, else of x's type.  kVec: x and the result lie on 4 values.
template <class X, int kDim, bool kE4m3, bool kVec>
__global__ void __launch_bounds__(kRotateThreads) norm_rotate_kernel(const __grid_constant__ NormRotateParams p)
{
    constexpr int kLanes = kDim / 8;
    const uint32_t unit = blockIdx.x * (kRotateThreads / kLanes) + threadIdx.x / kLanes;  // token and heads
    const int lane = threadIdx.x % kLanes;
    const int units = p.units[0] + p.units[1];
    const bool there = unit < uint32_t(p.T * units);
    const int32_t t = there ? p.by_units.of(int32_t(unit)) : 0;
    int32_t part = there ? int32_t(unit) - t * units : 0;
    const int which = part >= p.units[0];
    if (which) part -= p.units[0];
    const int h0 = part * p.per_unit, h1 = there ? min(h0 + p.per_unit, p.heads[which]) : h0;

    // ---- where the lane's two runs of four values lie; pair j is (a j, b j), or values 2 j and 2 j + 1 of them all
    const bool turns = 8 * lane < p.rotated;
    const bool apart = turns && !p.interleaved;
    const int at_a = apart ? 4 * lane : 8 * lane, at_b = apart ? p.rotated / 2 + 4 * lane : 8 * lane + 4;

    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // ---- the unit's first row (each one is loaded while the one before it is worked on)
    const X* const x = static_cast<const X*>(p.x[which]) + t * p.row_stride[which];
    float next_a[4] = {}, next_b[4] = {};
    auto load = [&](int h) {
        if (h >= h1) return;
        load4<X, kVec>(p.bounds, kMemRows + which, x + h * p.head_stride[which] + at_a, next_a);
        load4<X, kVec>(p.bounds, kMemRows + which, x + h * p.head_stride[which] + at_b, next_b);
    };
    load(h0);

    float c[4], s[4];  // of the pairs
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        c[j] = 1.0f;
        s[j] = 0.0f;
    }
    if (turns && there) {
        int64_t pos = 0;
        if (p.wide_positions) {
            const int64_t* const at = static_cast<const int64_t*>(p.positions) + t;
            if (in_bounds(p.bounds, kMemPositions, at, 8)) pos = *at;
        } else {
            const int32_t* const at = static_cast<const int32_t*>(p.positions) + t;
            if (in_bounds(p.bounds, kMemPositions, at, 4)) pos = *at;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float* const at = p.inv_freq + 4 * lane + j;
            const double f = in_bounds(p.bounds, kMemFreq, at, 4) ? double(*at) * 0.15915494309189533577 : 0.0;  // turns
            const uint64_t turn = uint64_t((f - floor(f)) * 18446744073709551616.0);
            // in halves of a turn, [-1, 1)
            const float half = float(int32_t((turn * uint64_t(pos)) >> 32)) * 0x1p-31f;
            sincospif(half, &s[j], &c[j]);
        }
    }
    // ---- the pairs' factors: out_a = x_a ca - x_b sb, out_b = x_b cb + x_a sa
    float ca[4], sa[4], cb[4], sb[4];
    const bool norm = p.weight[which] != nullptr;
    {
        float wa[4] = {1.0f, 1.0f, 1.0f, 1.0f}, wb[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if (norm) {
            if (p.weight_f32[which]) {
                load4<float, false>(p.bounds, kMemWeight + which, static_cast<const float*>(p.weight[which]) + at_a, wa);
                load4<float, false>(p.bounds, kMemWeight + which, static_cast<const float*>(p.weight[which]) + at_b, wb);
            } else {
                load4<X, false>(p.bounds, kMemWeight + which, static_cast<const X*>(p.weight[which]) + at_a, wa);
                load4<X, false>(p.bounds, kMemWeight + which, static_cast<const X*>(p.weight[which]) + at_b, wb);
            }
        }
        if (p.interleaved) {  // pairs (a0, a1), (a2, a3), (b0, b1), (b2, b3): as (a, b) each
            const float w[8] = {wa[0], wa[1], wa[2], wa[3], wb[0], wb[1], wb[2], wb[3]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                wa[j] = w[2 * j];
                wb[j] = w[2 * j + 1];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ca[j] = wa[j] * c[j];
            sa[j] = wa[j] * s[j];
            cb[j] = wb[j] * c[j];
            sb[j] = wb[j] * s[j];
        }
    }

    // all lanes of a warp go round together (they exchange sums); a group past its end does nothing
    for (int i = 0; i < p.per_unit; ++i) {
        const int h = h0 + i;
        const bool mine = h < h1;
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = next_a[j];
            b[j] = next_b[j];
        }
        load(h + 1);
        float by = 1.0f;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fmaf(a[j], a[j], fmaf(b[j], b[j], sum));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
        if (norm) by = rsqrtf(fmaf(sum, 1.0f / kDim, p.eps));
        if (p.interleaved) {
            const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = v[2 * j];
                b[j] = v[2 * j + 1];
            }
        }
        float ya[4], yb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (values that do not turn have nothing to do with one another: b may be infinite)
            ya[j] = by * (turns ? a[j] * ca[j] - b[j] * sb[j] : a[j] * ca[j]);
            yb[j] = by * (turns ? b[j] * cb[j] + a[j] * sa[j] : b[j] * cb[j]);
        }
        if (p.interleaved) {
            const float v[8] = {ya[0], yb[0], ya[1], yb[1], ya[2], yb[2], ya[3], yb[3]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ya[j] = v[j];
                yb[j] = v[4 + j];
            }
        }
        const int64_t to = t * p.out_row_stride[which] + h * p.out_head_stride[which];
        if constexpr (kE4m3) {
            float top = kTinyMax;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max_nan(top, max_nan(fabsf(ya[j]), fabsf(yb[j])));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
            const float inv = __fdiv_rn(kE4m3Max, top);
            auto pack = [&](const float (&y)[4]) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[0], inv), __fmul_rn(y[1], inv)),
                                                             __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[2], inv), __fmul_rn(y[3], inv)),
                                                             __NV_SATFINITE, __NV_E4M3);
                return lo | hi << 16;
            };
            if (mine) {
                uint8_t* const out = static_cast<uint8_t*>(p.out[which]) + to;
                const int kind = which ? kMemOut2 : kMemOut;
                if (in_bounds(p.bounds, kind, out + at_a, 4)) *reinterpret_cast<uint32_t*>(out + at_a) = pack(ya);
                if (in_bounds(p.bounds, kind, out + at_b, 4)) *reinterpret_cast<uint32_t*>(out + at_b) = pack(yb);
                float* const scale = p.out_scale[which] + int64_t(t) * p.heads[which] + h;
                if (lane == 0 && in_bounds(p.bounds, which ? kMemOutScale2 : kMemOutScale, scale, 4))
                    *scale = __fmul_rn(top, 1.0f / kE4m3Max);
            }
        } else if (mine) {
            X* const out = static_cast<X*>(p.out[which]) + to;
            store4<X, kVec>(p.bounds, which ? kMemOut2 : kMemOut, out + at_a, ya);
            store4<X, kVec>(p.bounds, which ? kMemOut2 : kMemOut, out + at_b, yb);
        }
    }
}

}  // namespace fp8mqa
