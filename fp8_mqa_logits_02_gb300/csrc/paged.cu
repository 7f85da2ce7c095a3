// Host side of the paged-cache entry points declared in include/fp8_mqa_logits.h: argument
// checks, the choice of kernel, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/fp8_mqa_logits.h"
#include "cache_kernels.cuh"
#include "paged_attention_kernel.cuh"
#include "paged_logits_kernel.cuh"

namespace fp8mqa {
namespace {

constexpr int kPagedMaxDevices = 64;
// Attention counters: a ring for direct launches, and one of its own for every launch captured
// into a CUDA graph (a graph's kernel keeps it for every replay).
constexpr uint32_t kAttnRing = 256, kAttnGraph = 1024;


struct PagedDevice {
    std::once_flag once;
    int status = FP8MQA_OK;
    int sm_count = 0;
    AttnCounters* counters = nullptr;  // kAttnRing + kAttnGraph, zero between launches
    std::atomic<uint32_t> ring{0}, graph{0};
};

PagedDevice g_paged[kPagedMaxDevices];

// CTAs of a full wave of the attention kernel.
int64_t attention_wave(int sm_count)
{
    return std::min<int64_t>(kAttnMaxCtas, int64_t(sm_count) * kAttnCtasPerSm);
}

template <int kType, int kDim>
bool attention_smem()
{
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return cudaFuncSetAttribute(paged_attention_kernel<kType, kDim, 1>, attr,
                                AttnShape<kType, kDim, 1>::kSmem) == cudaSuccess &&
           cudaFuncSetAttribute(paged_attention_kernel<kType, kDim, 2>, attr,
                                AttnShape<kType, kDim, 2>::kSmem) == cudaSuccess;
}

void init_paged(int dev, PagedDevice& st)
{
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&st.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        st.status = FP8MQA_ERR_CUDA;
        return;
    }
    if (major != 10 || minor != 3) {
        st.status = FP8MQA_ERR_ARCH;
        return;
    }
    if (!attention_smem<FP8MQA_E4M3, 64>() || !attention_smem<FP8MQA_E4M3, 128>() ||
        !attention_smem<FP8MQA_BF16, 64>() || !attention_smem<FP8MQA_BF16, 128>() ||
        !attention_smem<FP8MQA_F16, 64>() || !attention_smem<FP8MQA_F16, 128>()) {
        cudaGetLastError();
        st.status = FP8MQA_ERR_LAUNCH;
        return;
    }
    void* buf = nullptr;
    const size_t bytes = size_t(kAttnRing + kAttnGraph) * sizeof(AttnCounters);
    if (cudaMalloc(&buf, bytes) != cudaSuccess || cudaMemset(buf, 0, bytes) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(buf);
        st.status = FP8MQA_ERR_CUDA;
        return;
    }
    st.counters = static_cast<AttnCounters*>(buf);
}

PagedDevice* paged_device(int* err)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kPagedMaxDevices) {
        cudaGetLastError();
        *err = FP8MQA_ERR_CUDA;
        return nullptr;
    }
    PagedDevice& st = g_paged[dev];
    std::call_once(st.once, [dev, &st] { init_paged(dev, st); });
    *err = st.status;
    return st.status == FP8MQA_OK ? &st : nullptr;
}

bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t size_of(int32_t type) { return type == FP8MQA_E4M3 ? 1 : type == FP8MQA_F32 ? 4 : 2; }

// A cache argument: sizes, type, pointers, alignment.
int check_cache(const fp8mqa_cache* c)
{
    if (!c || c->pages < 0 || c->page_size < 1 || c->heads < 1) return FP8MQA_ERR_INVALID_ARG;
    if (c->type != FP8MQA_E4M3 && c->type != FP8MQA_BF16 && c->type != FP8MQA_F16)
        return FP8MQA_ERR_INVALID_ARG;
    if ((c->dim != 64 && c->dim != 128) || c->pages > INT32_MAX / int64_t(c->page_size))
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (c->pages > 0 && (!c->data || (c->type == FP8MQA_E4M3 && !c->scale)))
        return FP8MQA_ERR_INVALID_ARG;
    if ((c->type == FP8MQA_E4M3) != (c->scale != nullptr) && c->pages > 0)
        return FP8MQA_ERR_INVALID_ARG;
    // the stride of a dimension of one is never used
    const int64_t e = size_of(c->type);
    if (!on(c->data, 16) || !on(c->scale, 4) || (c->pages > 1 && c->page_stride * e % 16) ||
        (c->page_size > 1 && c->row_stride * e % 16) || (c->heads > 1 && c->head_stride * e % 16))
        return FP8MQA_ERR_MISALIGNED;
    return FP8MQA_OK;
}

PagedView view_of(const fp8mqa_cache& c)
{
    const int64_t e = size_of(c.type);
    PagedView v;
    v.data = static_cast<uint8_t*>(c.data);
    v.scale = c.scale;
    v.page_stride = c.page_stride * e;
    v.row_stride = c.row_stride * e;
    v.head_stride = c.head_stride * e;
    v.scale_page_stride = c.scale_page_stride;
    v.scale_row_stride = c.scale_row_stride;
    v.scale_head_stride = c.scale_head_stride;
    v.pages = int32_t(c.pages);
    v.page_size = c.page_size;
    v.heads = c.heads;
    return v;
}

// The counters of the launch being made, or null with *err set.
AttnCounters* attention_counters(PagedDevice& st, cudaStream_t s, int* err)
{
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {
        cudaGetLastError();
        *err = FP8MQA_ERR_CUDA;
        return nullptr;
    }
    if (cap == cudaStreamCaptureStatusNone)
        return st.counters + st.ring.fetch_add(1, std::memory_order_relaxed) % kAttnRing;
    const uint32_t i = st.graph.fetch_add(1, std::memory_order_relaxed);
    if (i >= kAttnGraph) {
        st.graph.store(kAttnGraph, std::memory_order_relaxed);
        *err = FP8MQA_ERR_CAPACITY;
        return nullptr;
    }
    return st.counters + kAttnRing + i;
}

int launched() { return cudaGetLastError() == cudaSuccess ? FP8MQA_OK : FP8MQA_ERR_LAUNCH; }

// CTAs of an attention launch: a full wave, or fewer where there are fewer tiles than that.  A
// CTA takes 8 heads, or 16 where a group has more than 8.
template <int kType, int kDim, int kNT>
void attention_launch(const PagedAttentionParams& p, int sm_count, cudaStream_t s)
{
    using S = AttnShape<kType, kDim, kNT>;
    const int64_t group = p.q_heads / p.k.heads;
    const int64_t longest =
        p.n_indices >= 0 ? p.n_indices : int64_t(p.table.cols) * p.k.page_size;
    const int64_t tiles = p.B * p.k.heads * ((group + S::kHeads - 1) / S::kHeads) *
                          std::max<int64_t>(1, (longest + S::kTile - 1) / S::kTile);
    const unsigned grid = unsigned(std::min(tiles, attention_wave(sm_count)));
    paged_attention_kernel<kType, kDim, kNT><<<grid, kAttnThreads, S::kSmem, s>>>(p);
}

template <int kType, int kDim>
void attention_heads(const PagedAttentionParams& p, int sm_count, cudaStream_t s)
{
    if (p.q_heads / p.k.heads <= 8)
        attention_launch<kType, kDim, 1>(p, sm_count, s);
    else
        attention_launch<kType, kDim, 2>(p, sm_count, s);
}

template <int kType>
void attention_dim(const PagedAttentionParams& p, int32_t dim, int sm_count, cudaStream_t s)
{
    if (dim == 64)
        attention_heads<kType, 64>(p, sm_count, s);
    else
        attention_heads<kType, 128>(p, sm_count, s);
}

}  // namespace
}  // namespace fp8mqa

extern "C" {

int fp8_mqa_cache_write(const int32_t* slots, int64_t T, int32_t x_type, const void* x,
                        int64_t x_row_stride, int64_t x_head_stride, const fp8mqa_cache* cache,
                        const void* x2, int64_t x2_row_stride, int64_t x2_head_stride,
                        const fp8mqa_cache* cache2, void* stream)
{
    using namespace fp8mqa;
    if (T < 0 || (x2 == nullptr) != (cache2 == nullptr)) return FP8MQA_ERR_INVALID_ARG;
    if (x_type != FP8MQA_BF16 && x_type != FP8MQA_F16 && x_type != FP8MQA_F32)
        return FP8MQA_ERR_INVALID_ARG;
    int rc = check_cache(cache);
    if (rc == FP8MQA_OK && cache2) rc = check_cache(cache2);
    if (rc != FP8MQA_OK) return rc;
    if (cache->type != FP8MQA_E4M3 ||
        (cache2 && (cache2->type != FP8MQA_E4M3 || cache2->page_size != cache->page_size ||
                    cache2->heads != cache->heads || cache2->dim != cache->dim)))
        return FP8MQA_ERR_INVALID_ARG;
    if (T * cache->heads >= int64_t(1) << 31) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return FP8MQA_OK;
    if (!slots || !x) return FP8MQA_ERR_INVALID_ARG;
    const uintptr_t e = uintptr_t(size_of(x_type));
    if (!on(slots, 4) || !on(x, e) || (x2 && !on(x2, e))) return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    if (!paged_device(&err)) return err;
    CacheWriteParams p;
    p.slots = slots;
    p.T = T;
    p.heads = cache->heads;
    p.dim = cache->dim;
    p.tensors = x2 ? 2 : 1;
    p.x[0] = x;
    p.x[1] = x2;
    p.row_stride[0] = x_row_stride;
    p.row_stride[1] = x2_row_stride;
    p.head_stride[0] = x_head_stride;
    p.head_stride[1] = x2_head_stride;
    p.cache[0] = view_of(*cache);
    p.cache[1] = view_of(cache2 ? *cache2 : *cache);
    const int64_t blocks = (T * p.heads * p.tensors + 7) / 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (x_type == FP8MQA_BF16)
        cache_write_kernel<__nv_bfloat16><<<unsigned(blocks), 256, 0, s>>>(p);
    else if (x_type == FP8MQA_F16)
        cache_write_kernel<__half><<<unsigned(blocks), 256, 0, s>>>(p);
    else
        cache_write_kernel<float><<<unsigned(blocks), 256, 0, s>>>(p);
    return launched();
}

int fp8_mqa_cache_read(const fp8mqa_cache* cache, const int32_t* table, int64_t table_stride,
                       int32_t table_cols, const int32_t* starts, int64_t B, int64_t total,
                       int32_t out_type, void* out, float* out_scale, void* stream)
{
    using namespace fp8mqa;
    const int rc = check_cache(cache);
    if (rc != FP8MQA_OK) return rc;
    if (cache->type != FP8MQA_E4M3 || B < 0 || total < 0 || table_cols < 0 || out_type < 0 ||
        out_type > FP8MQA_F32)
        return FP8MQA_ERR_INVALID_ARG;
    if (total * cache->heads >= int64_t(1) << 31 || B >= int64_t(1) << 31)
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (total == 0) return FP8MQA_OK;
    if (!starts || !out || (table_cols > 0 && B > 0 && !table) ||
        (out_type == FP8MQA_E4M3) != (out_scale != nullptr))
        return FP8MQA_ERR_INVALID_ARG;
    if (!on(table, 4) || !on(starts, 4) || !on(out, 16) || !on(out_scale, 4))
        return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    if (!paged_device(&err)) return err;
    CacheReadParams p;
    p.cache = view_of(*cache);
    p.table = {table, table_stride, table_cols};
    p.starts = starts;
    p.B = B;
    p.total = total;
    p.dim = cache->dim;
    p.out = out;
    p.out_scale = out_scale;
    const unsigned blocks = unsigned((total * cache->heads + 7) / 8);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (out_type == FP8MQA_E4M3)
        cache_read_kernel<uint8_t><<<blocks, 256, 0, s>>>(p);
    else if (out_type == FP8MQA_BF16)
        cache_read_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(p);
    else if (out_type == FP8MQA_F16)
        cache_read_kernel<__half><<<blocks, 256, 0, s>>>(p);
    else
        cache_read_kernel<float><<<blocks, 256, 0, s>>>(p);
    return launched();
}

int fp8_mqa_logits_paged(const uint8_t* q_fp8, const float* w, int64_t B, int32_t T, int32_t H,
                         int32_t D, const fp8mqa_cache* keys, const int32_t* table,
                         int64_t table_stride, int32_t table_cols, const int32_t* lens, float* out,
                         int64_t ld, int64_t N, int32_t clean_logits, void* stream)
{
    using namespace fp8mqa;
    if (B < 0 || T < 0 || N < 0 || ld < N || table_cols < 0 ||
        (clean_logits != 0 && clean_logits != 1))
        return FP8MQA_ERR_INVALID_ARG;
    if (H != kPagedHeads || D != kPagedDim) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    const int rc = check_cache(keys);
    if (rc != FP8MQA_OK) return rc;
    if (keys->type != FP8MQA_E4M3 || keys->heads != 1 || keys->dim != kPagedDim)
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (B * T > 65535 || N >= int64_t(1) << 30) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0 || T == 0 || N == 0) return FP8MQA_OK;
    if (!q_fp8 || !w || !lens || !out || (table_cols > 0 && !table)) return FP8MQA_ERR_INVALID_ARG;
    if (!on(q_fp8, 16) || !on(w, 16) || !on(table, 4) || !on(lens, 4) || !on(out, 4))
        return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    if (!paged_device(&err)) return err;
    PagedLogitsParams p;
    p.q = q_fp8;
    p.w = w;
    p.keys = view_of(*keys);
    p.table = {table, table_stride, table_cols};
    p.lens = lens;
    p.out = out;
    p.ld = ld;
    p.N = N;
    p.B = B;
    p.T = T;
    p.clean = clean_logits;
    paged_logits_kernel<<<dim3(unsigned((N + 127) / 128), unsigned(B * T)), 128, 0,
                          static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}

uint64_t fp8_mqa_attention_paged_workspace_bytes(int32_t q_heads, int32_t dim)
{
    using namespace fp8mqa;
    int err = FP8MQA_OK;
    if (q_heads < 1 || dim < 1) return 0;
    const PagedDevice* st = paged_device(&err);
    if (!st) return 0;
    // two partial results a CTA: heads x dim sums, and each head's m and l
    return 2 * uint64_t(attention_wave(st->sm_count)) * kAttnMaxHeads * uint64_t(dim + 2) *
           sizeof(float);
}

int fp8_mqa_attention_paged(const void* q, int32_t q_type, int64_t B, int32_t q_heads,
                            int64_t q_row_stride, int64_t q_head_stride, const fp8mqa_cache* k,
                            const fp8mqa_cache* v, const int32_t* table, int64_t table_stride,
                            int32_t table_cols, const int32_t* lens, const int32_t* indices,
                            int64_t indices_stride, int32_t n_indices, float sm_scale, void* out,
                            float* lse, void* workspace, uint64_t workspace_bytes, void* stream)
{
    using namespace fp8mqa;
    if (B < 0 || q_heads < 1 || table_cols < 0 || n_indices < -1 ||
        (q_type != FP8MQA_BF16 && q_type != FP8MQA_F16))
        return FP8MQA_ERR_INVALID_ARG;
    int rc = check_cache(k);
    if (rc == FP8MQA_OK) rc = check_cache(v);
    if (rc != FP8MQA_OK) return rc;
    if (k->type != v->type || k->page_size != v->page_size || k->heads != v->heads ||
        k->dim != v->dim || q_heads % k->heads != 0 ||
        (k->type != FP8MQA_E4M3 && k->type != q_type))
        return FP8MQA_ERR_INVALID_ARG;
    if (B > 65535) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0) return FP8MQA_OK;
    if (!q || !lens || !out || !workspace || (table_cols > 0 && !table) ||
        (n_indices > 0 && !indices))
        return FP8MQA_ERR_INVALID_ARG;
    if (!on(q, 16) || (B > 1 && q_row_stride % 8) || (q_heads > 1 && q_head_stride % 8) || !on(out, 16) || !on(lens, 4) ||
        !on(table, 4) || !on(indices, 4) || !on(lse, 4) || !on(workspace, 256))
        return FP8MQA_ERR_MISALIGNED;
    int err = FP8MQA_OK;
    PagedDevice* st = paged_device(&err);
    if (!st) return err;
    if (workspace_bytes < fp8_mqa_attention_paged_workspace_bytes(q_heads, k->dim))
        return FP8MQA_ERR_INVALID_ARG;
    PagedAttentionParams p;
    p.q = q;
    p.q_row_stride = q_row_stride;
    p.q_head_stride = q_head_stride;
    p.k = view_of(*k);
    p.v = view_of(*v);
    p.k.pages = p.v.pages = p.k.pages < p.v.pages ? p.k.pages : p.v.pages;
    p.table = {table, table_stride, table_cols};
    p.lens = lens;
    p.indices = indices;
    p.indices_stride = indices_stride;
    p.n_indices = n_indices;
    p.q_heads = q_heads;
    p.B = B;
    p.sm_scale = sm_scale;
    p.out = out;
    p.lse = lse;
    p.q_bf16 = q_type == FP8MQA_BF16;
    p.partial = static_cast<float*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.counters = attention_counters(*st, s, &err);
    if (!p.counters) return err;
    if (k->type == FP8MQA_E4M3)
        attention_dim<FP8MQA_E4M3>(p, k->dim, st->sm_count, s);
    else if (k->type == FP8MQA_BF16)
        attention_dim<FP8MQA_BF16>(p, k->dim, st->sm_count, s);
    else
        attention_dim<FP8MQA_F16>(p, k->dim, st->sm_count, s);
    return launched();
}

}  // extern "C"
