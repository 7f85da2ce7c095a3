// Writing rows into a paged E4M3 cache, and packing them back.
#pragma once

#include "paged_common.cuh"

namespace fp8mqa {

struct CacheWriteParams {
    const int32_t* slots;
    int64_t T;
    int32_t heads, dim, tensors;
    const void* x[2];
    int64_t row_stride[2], head_stride[2];
    PagedView cache[2];
};

// One warp per (tensor, token, head).
template <class X>
__global__ void cache_write_kernel(CacheWriteParams p)
{
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= p.T * p.heads * p.tensors) return;
    const int which = int(row / (p.T * p.heads));
    const int64_t t = row / p.heads % p.T;
    const int h = int(row % p.heads);
    const PagedView& c = p.cache[which];
    const int32_t slot = p.slots[t];
    if (slot < 0 || slot >= int64_t(c.pages) * c.page_size) return;
    const X* x = static_cast<const X*>(p.x[which]) + t * p.row_stride[which] +
                 h * p.head_stride[which];
    float a = kTinyMax;
    for (int d = lane; d < p.dim; d += 32) a = max_nan(a, fabsf(to_float(x[d])));
    for (int o = 16; o > 0; o /= 2) a = max_nan(a, __shfl_xor_sync(~0u, a, o));
    const float inv = __fdiv_rn(kE4m3Max, a);
    const int32_t page = slot / c.page_size, r = slot % c.page_size;
    uint8_t* out = c.data + page * c.page_stride + r * c.row_stride + h * c.head_stride;
    for (int d = lane; d < p.dim; d += 32)
        out[d] = __nv_cvt_float_to_fp8(__fmul_rn(to_float(x[d]), inv), __NV_SATFINITE, __NV_E4M3);
    if (lane == 0)
        c.scale[page * c.scale_page_stride + r * c.scale_row_stride + h * c.scale_head_stride] =
            __fmul_rn(a, 1.0f / kE4m3Max);
}

struct CacheReadParams {
    PagedView cache;
    PageTable table;
    const int32_t* starts;
    int64_t B, total;
    int32_t dim;
    void* out;
    float* out_scale;
};

// The sequence of output row r: the last b with starts[b] <= r (B where r is past the end).
__device__ __forceinline__ int64_t sequence_of(const int32_t* starts, int64_t B, int64_t r)
{
    int64_t lo = 0, hi = B + 1;  // the first b with starts[b] > r lies in [lo, hi]
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (__ldg(starts + mid) > r) hi = mid;
        else lo = mid + 1;
    }
    return lo - 1;
}

// One warp per output row and head.
template <class Out>
__global__ void cache_read_kernel(CacheReadParams p)
{
    const PagedView& c = p.cache;
    const int64_t at = int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (at >= p.total * c.heads) return;
    const int64_t r = at / c.heads;
    const int h = int(at % c.heads);
    const int64_t b = sequence_of(p.starts, p.B, r);
    int32_t page = 0, row = 0;
    const bool there =
        b >= 0 && b < p.B && locate(c, p.table, b, int32_t(r - __ldg(p.starts + b)), &page, &row);
    const uint8_t* src = c.data + page * c.page_stride + row * c.row_stride + h * c.head_stride;
    const float s = there ? c.scale[page * c.scale_page_stride + row * c.scale_row_stride +
                                    h * c.scale_head_stride]
                          : 0.0f;
    Out* out = static_cast<Out*>(p.out) + at * p.dim;
    for (int d = lane; d < p.dim; d += 32) {
        const uint8_t v = there ? src[d] : uint8_t(0);
        if constexpr (sizeof(Out) == 1)
            out[d] = v;
        else
            out[d] = there ? from_float<Out>(__fmul_rn(e4m3_to_float(v), s)) : from_float<Out>(0.0f);
    }
    if (sizeof(Out) == 1 && lane == 0) p.out_scale[at] = s;
}

}  // namespace fp8mqa
