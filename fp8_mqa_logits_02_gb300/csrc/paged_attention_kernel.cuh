// Attention of one new token per row over a paged cache, all of it or selected positions.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"

namespace fp8mqa {

struct PagedAttentionParams {
    const void* q;
    int64_t q_row_stride, q_head_stride;  // elements
    PagedView k, v;
    PageTable table;
    const int32_t* lens;
    const int32_t* indices;
    int64_t indices_stride;
    int32_t n_indices;
    int32_t q_heads;
    int64_t B;
    float sm_scale;
    void* out;
    float* lse;
};

// One block of 4 warps per (row, query head); each warp takes every fourth position with a
// running maximum and sum, and the warps' results are joined at the end.
template <class Q, class C, int kDim>
__global__ void paged_attention_kernel(PagedAttentionParams p)
{
    constexpr int kWarps = 4, kPer = kDim / 32;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kDim];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t b = blockIdx.y;
    const int h = blockIdx.x, g = h / (p.q_heads / p.k.heads);
    const Q* q = static_cast<const Q*>(p.q) + b * p.q_row_stride + h * p.q_head_stride;
    float qr[kPer], o[kPer] = {}, m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) qr[i] = to_float(q[lane + 32 * i]) * p.sm_scale;
    const int64_t cap = int64_t(p.table.cols) * p.k.page_size;
    const int32_t len = int32_t(min(int64_t(p.lens[b]), cap));
    const int32_t count = p.n_indices >= 0 ? p.n_indices : len;
    for (int32_t i = warp; i < count; i += kWarps) {
        const int32_t n = p.n_indices >= 0 ? __ldg(p.indices + b * p.indices_stride + i) : i;
        int32_t page, row;
        if (n < 0 || n >= len || !locate(p.k, p.table, b, n, &page, &row)) continue;
        const C* k = reinterpret_cast<const C*>(p.k.data + page * p.k.page_stride +
                                                row * p.k.row_stride + g * p.k.head_stride);
        const C* v = reinterpret_cast<const C*>(p.v.data + page * p.v.page_stride +
                                                row * p.v.row_stride + g * p.v.head_stride);
        float ks = 1.0f, vs = 1.0f;
        if (sizeof(C) == 1) {
            ks = p.k.scale[page * p.k.scale_page_stride + row * p.k.scale_row_stride +
                           g * p.k.scale_head_stride];
            vs = p.v.scale[page * p.v.scale_page_stride + row * p.v.scale_row_stride +
                           g * p.v.scale_head_stride];
        }
        float x = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) x = fmaf(qr[j], to_float(k[lane + 32 * j]), x);
        for (int s = 16; s > 0; s /= 2) x += __shfl_xor_sync(~0u, x, s);
        x *= ks;
        const float top = fmaxf(m, x);
        const float c = m == -CUDART_INF_F ? 0.0f : __expf(m - top), e = __expf(x - top);
        l = l * c + e;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            o[j] = o[j] * c + e * vs * to_float(v[lane + 32 * j]);
        m = top;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) s_o[warp][lane + 32 * j] = o[j];
    __syncthreads();
    float top = -CUDART_INF_F;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    float total = 0.0f, c[kWarps];
    for (int w = 0; w < kWarps; ++w) {
        c[w] = s_m[w] == -CUDART_INF_F ? 0.0f : __expf(s_m[w] - top);
        total += c[w] * s_l[w];
    }
    const int64_t at = b * p.q_heads + h;
    for (int d = threadIdx.x; d < kDim; d += kWarps * 32) {
        float sum = 0.0f;
        for (int w = 0; w < kWarps; ++w) sum += c[w] * s_o[w][d];
        static_cast<Q*>(p.out)[at * kDim + d] = from_float<Q>(total > 0.0f ? sum / total : 0.0f);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[at] = total > 0.0f ? top + logf(total) : -CUDART_INF_F;
}

}  // namespace fp8mqa
