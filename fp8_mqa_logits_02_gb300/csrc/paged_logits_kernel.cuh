// The indexer logits of each sequence's newest tokens, read straight from the cache's pages.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"

namespace fp8mqa {

struct PagedLogitsParams {
    const uint8_t* q;
    const float* w;
    PagedView keys;
    PageTable table;
    const int32_t* lens;
    float* out;
    int64_t ld, N, B;
    int32_t T, clean;
};

constexpr int kPagedHeads = 32, kPagedDim = 128;

// One thread per (row, key), the row's queries in shared memory.
__global__ void paged_logits_kernel(PagedLogitsParams p)
{
    __shared__ float q[kPagedHeads * kPagedDim], w[kPagedHeads];
    const int64_t row = blockIdx.y, b = row / p.T;
    const int t = int(row % p.T);
    for (int i = threadIdx.x; i < kPagedHeads * kPagedDim; i += blockDim.x)
        q[i] = e4m3_to_float(p.q[row * kPagedHeads * kPagedDim + i]);
    if (threadIdx.x < kPagedHeads) w[threadIdx.x] = p.w[row * kPagedHeads + threadIdx.x];
    __syncthreads();
    const int64_t n = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (n >= p.N) return;
    const int64_t end = int64_t(p.lens[b]) - (p.T - 1 - t);
    int32_t page = 0, r = 0;
    if (n >= end) {
        if (p.clean) p.out[row * p.ld + n] = -CUDART_INF_F;
        return;
    }
    if (!locate(p.keys, p.table, b, int32_t(n), &page, &r)) {
        p.out[row * p.ld + n] = -CUDART_INF_F;
        return;
    }
    float k[kPagedDim];
    const uint8_t* src = p.keys.data + page * p.keys.page_stride + r * p.keys.row_stride;
#pragma unroll
    for (int d = 0; d < kPagedDim; ++d) k[d] = e4m3_to_float(src[d]);
    float sum = 0.0f;
    for (int h = 0; h < kPagedHeads; ++h) {
        float dot = 0.0f;
#pragma unroll
        for (int d = 0; d < kPagedDim; ++d) dot = fmaf(q[h * kPagedDim + d], k[d], dot);
        sum = fmaf(fmaxf(dot, 0.0f), w[h], sum);
    }
    p.out[row * p.ld + n] =
        sum * p.keys.scale[page * p.keys.scale_page_stride + r * p.keys.scale_row_stride];
}

}  // namespace fp8mqa
