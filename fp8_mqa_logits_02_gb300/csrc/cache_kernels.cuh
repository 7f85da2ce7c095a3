// Writing rows into a paged E4M3 cache, and packing them back.  Both move bytes and are bound by
// them, so the wider side goes 16 bytes a lane, side by side.
#pragma once

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

struct CacheReadParams {
    PagedView cache;
    PageTable table;
    FastDiv by_heads;
    const int32_t* starts;
    int64_t B, total;
    int32_t block_rows;  // output rows of a block, kReadRows at most
    void* out;
    float* out_scale;
    PagedBounds bounds;
};
constexpr int kReadRows = 128;

constexpr int kReadPieces = 4;  // pieces of 16 bytes of output that a thread has under way

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
// threads copy their pieces, which are contiguous in the output.  66 thousand rows x 8 heads to bfloat16
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

}  // namespace fp8mqa
