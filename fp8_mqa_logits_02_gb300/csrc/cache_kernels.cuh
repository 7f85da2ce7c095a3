// Writing rows into a paged E4M3 cache, and packing them back.  Both move bytes and are bound by
// them, so the wider side goes 16 bytes a lane, side by side.
#pragma once

#include <type_traits>

#include "paged_common.cuh"

namespace fp8mqa {

constexpr int kCacheThreads = 256;

struct CacheWriteParams {
    const int32_t* slots;
    int64_t T;
    int32_t heads;
    FastDiv by_heads, by_page;
    const void* x[2];
    int64_t row_stride[2], head_stride[2];
    PagedView cache[2];
    int32_t alike;  // the two caches' strides
    PagedBounds bounds;
};

// Lane c's 16 values of a row as floats: pieces c, c + kLanes, ... of 16 bytes, so that the lanes of a
// row load (and store) side by side.  kVec: x lies on 16 bytes.
template <class X, bool kVec, int kLanes>
__device__ __forceinline__ void load16(const PagedBounds& bounds, int kind, const X* x, int c, float (&v)[16])
{
    constexpr int kPer = 16 / sizeof(X);
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
        alignas(16) X raw[kPer];
        const X* const at = x + (c + i * kLanes) * kPer;
        if (!in_bounds(bounds, kind, at, 16)) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) raw[j] = from_float<X>(0.0f);
        } else if constexpr (kVec) {
            *reinterpret_cast<uint4*>(raw) = __ldcs(reinterpret_cast<const uint4*>(at));
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) raw[j] = at[j];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[i * kPer + j] = to_float(raw[j]);
    }
}

// A group of kDim / 16 lanes per (token, head) quantises that row of each tensor: the row's loads do
// not wait for its slot, and keys and values share the slot.  16384 tokens x 8 heads of bfloat16 keys and
// values (102 MB): 16.9 us, 6.0 TB/s of 6.7; a warp a row, value by value, took 95.
template <class X, int kDim, bool kVec, int kTensors>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const __grid_constant__ CacheWriteParams p)
{
    constexpr int kLanes = kDim / 16, kPer = 16 / sizeof(X);
    const uint32_t at = blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;  // token and head
    const int c = threadIdx.x % kLanes;
    const bool row = at < uint32_t(p.T * p.heads);
    const int32_t t = row ? p.by_heads.of(int32_t(at)) : 0, h = row ? int32_t(at) - t * p.heads : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t slot = row && in_bounds(p.bounds, kMemSlots, p.slots + t, 4) ? p.slots[t] : -1;
    float v[kTensors][16];
#pragma unroll
    for (int i = 0; i < kTensors; ++i)
        load16<X, kVec, kLanes>(
            p.bounds, kMemRows + i,
            static_cast<const X*>(p.x[i]) + t * p.row_stride[i] + h * p.head_stride[i], c, v[i]);
    const int32_t page = p.by_page.of(max(slot, 0)), r = slot - page * p.cache[0].page_size;
#pragma unroll
    for (int i = 0; i < kTensors; ++i) {
        float a = kTinyMax;
#pragma unroll
        for (int j = 0; j < 16; ++j) a = max_nan(a, fabsf(v[i][j]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) a = max_nan(a, __shfl_xor_sync(~0u, a, o));
        const PagedView& cache = p.cache[i];
        if (slot < 0 || page >= cache.pages) continue;
        const float inv = __fdiv_rn(kE4m3Max, a);
        uint32_t out[4];  // value j is byte j
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(v[i][4 * j], inv), __fmul_rn(v[i][4 * j + 1], inv)),
                __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(v[i][4 * j + 2], inv), __fmul_rn(v[i][4 * j + 3], inv)),
                __NV_SATFINITE, __NV_E4M3);
            out[j] = lo | hi << 16;
        }
        uint8_t* const to = cache.data + page * cache.page_stride + r * cache.row_stride +
                            h * cache.head_stride + c * kPer;
        if constexpr (kPer == 8) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (in_bounds(p.bounds, kMemData + i, to + 8 * kLanes * j, 8))
                    *reinterpret_cast<uint2*>(to + 8 * kLanes * j) = make_uint2(out[2 * j], out[2 * j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in_bounds(p.bounds, kMemData + i, to + 4 * kLanes * j, 4))
                    *reinterpret_cast<uint32_t*>(to + 4 * kLanes * j) = out[j];
        }
        float* const to_scale = cache.scale + page * cache.scale_page_stride +
                                r * cache.scale_row_stride + h * cache.scale_head_stride;
        if (c == 0 && in_bounds(p.bounds, kMemScale + i, to_scale, 4))
            *to_scale = __fmul_rn(a, 1.0f / kE4m3Max);
    }
}

// The same for E2M1 caches: a lane has a group of 16 values side by side, so that its scale and values need
// nothing of other lanes but the row's maximum.  With a the row's maximum and m the group's:
//     G = e4m3(448 m / a);  data = e2m1(2688 x / (G a));  scale = a / 2688
// What the values and m are divided by is exact, and the quotients are rounded as a division is, so that
// ties of 16-bit inputs fall as in real arithmetic: rows are first scaled by a power of two that brings a to
// [1, 2), and then, with y the correctly rounded reciprocal of b, q = y n is off by r = n - q b, which a fused
// multiply-add gives exactly, and q + y r is the quotient rounded (P. Markstein, IBM J. Res. Dev. 34, 1990).
// 16 thousand tokens x 8 heads of bfloat16 keys and values (86 MB): 18.5 us, 4.7 TB/s of 6.8 (fp32 rows, 159 MB:
// 23.4).  The quotients are 2.5 us of it, with some 200 instructions for 16 values (65 % of the issue slots), and loads
// are what warps wait for most: 60 registers for both tensors leave 41 % of the warps.
template <class X>
struct alignas(16) Group {
    X v[kGroup];
};

// kVec: the group lies on 32 bytes.
template <class X, bool kVec>
__device__ __forceinline__ Group<X> load_group(const PagedBounds& bounds, int kind, const X* x)
{
    constexpr int kPer = 32 / sizeof(X);
    Group<X> r;
#pragma unroll
    for (int j = 0; j < kGroup; j += kPer) {
        if (!in_bounds(bounds, kind, x + j, 32)) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) r.v[j + k] = from_float<X>(0.0f);
        } else if constexpr (kVec) {
            uint32_t* const w = reinterpret_cast<uint32_t*>(&r.v[j]);
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(x + j));
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k) r.v[j + k] = x[j + k];
        }
    }
    return r;
}

// The largest magnitude of a group, NaN if there is one; 16-bit values go two at a time.
__device__ __forceinline__ float largest(const Group<float>& x)
{
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) m = max_nan(m, fabsf(x.v[j]));
    return m;
}
template <class X>
__device__ __forceinline__ float largest(const Group<X>& x)
{
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(&x);
    uint32_t m = w[0];
#pragma unroll
    for (int j = 1; j < kGroup / 2; ++j) {
        if constexpr (std::is_same_v<X, __nv_bfloat16>)
            asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j]));
        else
            asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j]));
    }
    const X* const two = reinterpret_cast<const X*>(&m);
    return max_nan(fabsf(to_float(two[0])), fabsf(to_float(two[1])));
}

// n / b, given the correctly rounded 1 / b.
__device__ __forceinline__ float quotient(float n, float b, float reciprocal)
{
    const float q = n * reciprocal;
    return fmaf(fmaf(-q, b, n), reciprocal, q);
}

// x by / b of two values at a time, given -b and the correctly rounded 1 / b, twice each.
__device__ __forceinline__ void quotients(float& x0, float& x1, uint64_t by, uint64_t minus_b, uint64_t reciprocal)
{
    asm("{\n\t.reg .b64 n, q, r;\n\tmov.b64 n, {%0, %1};\n\tmul.rn.f32x2 n, n, %2;\n\tmul.rn.f32x2 q, n, %4;\n\t"
        "fma.rn.f32x2 r, q, %3, n;\n\tfma.rn.f32x2 q, r, %4, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "l"(by), "l"(minus_b), "l"(reciprocal));
}
__device__ __forceinline__ uint64_t both(float x)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}

template <class X, int kDim, bool kVec, int kTensors>
__global__ void __launch_bounds__(kCacheThreads) cache_write4_kernel(const __grid_constant__ CacheWriteParams p)
{
    constexpr int kLanes = kDim / kGroup;
    const uint32_t at = blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;  // token and head
    const int c = threadIdx.x % kLanes;
    const bool row = at < uint32_t(p.T * p.heads);
    const int32_t t = row ? p.by_heads.of(int32_t(at)) : 0, h = row ? int32_t(at) - t * p.heads : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t slot = row && in_bounds(p.bounds, kMemSlots, p.slots + t, 4) ? p.slots[t] : -1;
    Group<X> raw[kTensors];
#pragma unroll
    for (int i = 0; i < kTensors; ++i)
        raw[i] = load_group<X, kVec>(p.bounds, kMemRows + i, static_cast<const X*>(p.x[i]) + t * p.row_stride[i] +
                                                                 h * p.head_stride[i] + c * kGroup);
    int64_t at_data = 0, at_group = 0, at_scale = 0;
    const int32_t page = p.by_page.of(max(slot, 0)), r = slot - page * p.cache[0].page_size;
#pragma unroll
    for (int i = 0; i < kTensors; ++i) {
        const float m = largest(raw[i]);
        float a = max_nan(m, kTinyMax);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) a = max_nan(a, __shfl_xor_sync(~0u, a, o));
        const PagedView& cache = p.cache[i];
        // (before the look at the page: the second cache may have pages that the first has not)
        if (i == 0 || !p.alike) {
            at_data = page * cache.page_stride + r * cache.row_stride + h * cache.head_stride + c * 8;
            at_group = page * cache.group_page_stride + r * cache.group_row_stride + h * cache.group_head_stride + c;
            at_scale = page * cache.scale_page_stride + r * cache.scale_row_stride + h * cache.scale_head_stride;
        }
        if (slot < 0 || page >= cache.pages) continue;
        // 2^-e of a in [2^e, 2^(e + 1)); the largest ones, and what is not finite, take 2^-126
        const float down = __uint_as_float((254u - min(__float_as_uint(a) >> 23, 253u)) << 23);
        const float top = a * down;
        const uint32_t g = __nv_cvt_float_to_fp8(quotient(m * down * kE4m3Max, top, __frcp_rn(top)), __NV_SATFINITE, __NV_E4M3);
        const float b = __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(g), __NV_E4M3))) * top;
        const float y = b > 0.0f ? __frcp_rn(b) : 0.0f;
        const uint64_t by2 = both(down * kE2m1Top), b2 = both(-b), y2 = both(y);
        float v[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; j += 2) {
            v[j] = to_float(raw[i].v[j]);
            v[j + 1] = to_float(raw[i].v[j + 1]);
            quotients(v[j], v[j + 1], by2, b2, y2);
        }
        uint8_t* const to = cache.data + at_data;
        if (in_bounds(p.bounds, kMemData + i, to, 8))
            *reinterpret_cast<uint2*>(to) = make_uint2(e2m1_of(v), e2m1_of(v + 8));
        uint8_t* const to_group = cache.groups + at_group;
        if (in_bounds(p.bounds, kMemGroups + i, to_group, 1)) *to_group = uint8_t(g);
        float* const to_scale = cache.scale + at_scale;
        // (an infinity would leave infinities where it is not among the values that round to 0)
        if (c == 0 && in_bounds(p.bounds, kMemScale + i, to_scale, 4))
            *to_scale = a <= 3.402823466e38f ? __fmul_rn(a, 1.0f / kE2m1Top) : __uint_as_float(0x7FC00000u);
    }
}

struct CacheReadParams {
    PagedView cache;
    PageTable table;
    FastDiv by_heads;
    const int32_t* starts;
    int64_t B, total;
    int32_t block_rows;  // output rows of a block, kReadRows at most
    void* out;
    float* out_scale;
    int32_t aligned32;  // out lies on 32 bytes
    PagedBounds bounds;
};
constexpr int kReadRows = 128;

constexpr int kReadPieces = 4;  // pieces of 16 bytes of output that a thread has under way
constexpr int kReadPieces4 = 1;  // groups of an E2M1 cache

// The sequence of output row r: the last b with starts[b] <= r (B where r is past the end).
template <class Starts>
__device__ __forceinline__ int64_t sequence_of(const Starts& starts, int64_t B, int64_t r)
{
    int64_t lo = 0, hi = B + 1;  // the first b with starts[b] > r lies in [lo, hi]
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (starts(mid) > r) hi = mid;
        else lo = mid + 1;
    }
    return lo - 1;
}

// A block packs block_rows consecutive output rows: first a thread a row finds where it lies, then all
// threads copy their pieces, which are contiguous in the output.  75 thousand rows x 8 heads to bfloat16
// (234 MB): 39 us, 5.9 TB/s of 6.7; a warp a row took 182, eight pieces under way instead of four 42.
template <class Out, int kDim>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const __grid_constant__ CacheReadParams p)
{
    __shared__ int64_t s_data[kReadRows], s_scale[kReadRows];  // offsets; -1: not there
    const PagedView& c = p.cache;
    const int64_t r0 = int64_t(blockIdx.x) * p.block_rows;
    const int rows = int(min(int64_t(p.block_rows), p.total - r0));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < rows) {
        auto starts = [&](int64_t b) { return in_bounds(p.bounds, kMemLens, p.starts + b, 4) ? p.starts[b] : 0; };
        const int64_t r = r0 + threadIdx.x, b = sequence_of(starts, p.B, r);
        int32_t page = 0, row = 0;
        const bool there =
            b >= 0 && b < p.B && locate(p.bounds, c, p.table, b, int32_t(r - starts(b)), &page, &row);
        s_data[threadIdx.x] = there ? page * c.page_stride + row * c.row_stride : -1;
        s_scale[threadIdx.x] = page * c.scale_page_stride + row * c.scale_row_stride;
    }
    __syncthreads();
    constexpr int kPer = 16 / sizeof(Out), kLanes = kDim / kPer;
    const int n = rows * c.heads * kLanes;
    uint4* const out = reinterpret_cast<uint4*>(static_cast<Out*>(p.out) + r0 * c.heads * kDim);
    for (int i0 = threadIdx.x; i0 < n; i0 += kReadPieces * kCacheThreads) {
        uint32_t x[kReadPieces][kPer / 4];
        float by[kReadPieces];
#pragma unroll
        for (int j = 0; j < kReadPieces; ++j) {
            const int i = i0 + j * kCacheThreads, at = i / kLanes;
#pragma unroll
            for (int k = 0; k < kPer / 4; ++k) x[j][k] = 0u;
            by[j] = 0.0f;
            if (i < n) {
                const int row = p.by_heads.of(at), h = at - row * c.heads;
                const int64_t off = s_data[row];
                const uint8_t* const src = c.data + off + h * c.head_stride + i % kLanes * kPer;
                const float* const src_scale = c.scale + s_scale[row] + h * c.scale_head_stride;
                if (off >= 0 && in_bounds(p.bounds, kMemData, src, kPer) &&
                    in_bounds(p.bounds, kMemScale, src_scale, 4)) {
                    if constexpr (kPer == 16) {
                        const uint4 y = __ldcs(reinterpret_cast<const uint4*>(src));
                        x[j][0] = y.x;
                        x[j][1] = y.y;
                        x[j][2] = y.z;
                        x[j][3] = y.w;
                    } else if constexpr (kPer == 8) {
                        const uint2 y = __ldcs(reinterpret_cast<const uint2*>(src));
                        x[j][0] = y.x;
                        x[j][1] = y.y;
                    } else {
                        x[j][0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
                    }
                    by[j] = *src_scale;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kReadPieces; ++j) {
            const int i = i0 + j * kCacheThreads;
            if (i >= n) break;
            if (!in_bounds(p.bounds, kMemOut, out + i, 16)) continue;
            if constexpr (kPer == 16) {
                out[i] = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
                float* const to_scale = p.out_scale + r0 * c.heads + i / kLanes;
                if (i % kLanes == 0 && in_bounds(p.bounds, kMemOutScale, to_scale, 4)) *to_scale = by[j];
            } else {
                // a row that is not there has zeros and a zero scale
                alignas(16) Out y[kPer];
#pragma unroll
                for (int k = 0; k < kPer / 4; ++k) {
                    uint32_t two[2];
                    f16_of_e4m3(x[j][k], &two[0], &two[1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two[h]));
                        y[4 * k + 2 * h] = from_float<Out>(__fmul_rn(f.x, by[j]));
                        y[4 * k + 2 * h + 1] = from_float<Out>(__fmul_rn(f.y, by[j]));
                    }
                }
                out[i] = *reinterpret_cast<const uint4*>(y);
            }
        }
    }
}

// 32 bytes in one store where they lie on 32, else in two.
__device__ __forceinline__ void store32(void* to, const uint32_t* w, bool aligned)
{
    if (aligned)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        static_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// The same from an E2M1 cache: a piece is a group, 16 values.  75 thousand rows x 8 heads to bfloat16 (201 MB): 36.8 us
// (47 with two stores of 16 bytes instead of one of 32; 39 with two groups a thread under way, which leaves fewer
// threads an SM, 58 with eight).
template <class Out, int kDim>
__global__ void __launch_bounds__(kCacheThreads) cache_read4_kernel(const __grid_constant__ CacheReadParams p)
{
    __shared__ int64_t s_data[kReadRows], s_scale[kReadRows], s_group[kReadRows];  // offsets; s_data -1: not there
    const PagedView& c = p.cache;
    const int64_t r0 = int64_t(blockIdx.x) * p.block_rows;
    const int rows = int(min(int64_t(p.block_rows), p.total - r0));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < rows) {
        auto starts = [&](int64_t b) { return in_bounds(p.bounds, kMemLens, p.starts + b, 4) ? p.starts[b] : 0; };
        const int64_t r = r0 + threadIdx.x, b = sequence_of(starts, p.B, r);
        int32_t page = 0, row = 0;
        const bool there =
            b >= 0 && b < p.B && locate(p.bounds, c, p.table, b, int32_t(r - starts(b)), &page, &row);
        s_data[threadIdx.x] = there ? page * c.page_stride + row * c.row_stride : -1;
        s_scale[threadIdx.x] = page * c.scale_page_stride + row * c.scale_row_stride;
        s_group[threadIdx.x] = page * c.group_page_stride + row * c.group_row_stride;
    }
    __syncthreads();
    constexpr int kLanes = kDim / kGroup;
    const int n = rows * c.heads * kLanes;
    Out* const out = static_cast<Out*>(p.out) + r0 * c.heads * kDim;
    for (int i0 = threadIdx.x; i0 < n; i0 += kReadPieces4 * kCacheThreads) {
        uint2 x[kReadPieces4];
        float by[kReadPieces4];
        uint32_t g[kReadPieces4];
#pragma unroll
        for (int j = 0; j < kReadPieces4; ++j) {
            const int i = i0 + j * kCacheThreads, at = i / kLanes;
            x[j] = make_uint2(0u, 0u);
            by[j] = 0.0f;
            g[j] = 0u;
            if (i < n) {
                const int row = p.by_heads.of(at), h = at - row * c.heads;
                const int64_t off = s_data[row];
                const uint8_t* const src = c.data + off + h * c.head_stride + i % kLanes * 8;
                const uint8_t* const src_group = c.groups + s_group[row] + h * c.group_head_stride + i % kLanes;
                const float* const src_scale = c.scale + s_scale[row] + h * c.scale_head_stride;
                if (off >= 0 && in_bounds(p.bounds, kMemData, src, 8) && in_bounds(p.bounds, kMemScale, src_scale, 4) &&
                    in_bounds(p.bounds, kMemGroups, src_group, 1)) {
                    x[j] = __ldcs(reinterpret_cast<const uint2*>(src));
                    g[j] = *src_group;
                    by[j] = *src_scale;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kReadPieces4; ++j) {
            const int i = i0 + j * kCacheThreads;
            if (i >= n) break;
            const uint32_t group = f16x2_of_e4m3x2(g[j] * 0x101u);
            uint32_t h[8];
            f16_of_e2m1(x[j].x, *reinterpret_cast<uint32_t(*)[4]>(h));
            f16_of_e2m1(x[j].y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
            alignas(16) Out y[kGroup];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t two = mul_f16x2(h[k], group);  // exact
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
                y[2 * k] = from_float<Out>(__fmul_rn(f.x, by[j]));
                y[2 * k + 1] = from_float<Out>(__fmul_rn(f.y, by[j]));
            }
            Out* const to = out + int64_t(i) * kGroup;
#pragma unroll
            for (int k = 0; k < int(kGroup * sizeof(Out) / 32); ++k)
                if (in_bounds(p.bounds, kMemOut, to + k * (32 / sizeof(Out)), 32))
                    store32(to + k * (32 / sizeof(Out)), reinterpret_cast<const uint32_t*>(y) + 8 * k, p.aligned32);
        }
    }
}

}  // namespace fp8mqa
