// Host side of a serving step's other entry points declared in include/fp8_mqa_logits.h: page tables,
// and norms with rotation.  Argument checks, the choice of kernel, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/fp8_mqa_logits.h"
#include "norm_rotate_kernel.cuh"
#include "overlap.h"
#include "pages_kernel.cuh"
#include "paged_launch.cuh"

namespace fp8mqa {
namespace {

size_t pages_smem_bytes(int32_t B) { return 4 * size_t(B + 1) * sizeof(int32_t); }

// A cluster for what it has the threads for, else a CTA for each kPagesTokens tokens and then the lengths.  By the rows
// for new tokens alone, which the host knows; pages that come and go take what CTAs there are.
constexpr int64_t kPagesTokens = 4 * kPagesThreads;
constexpr unsigned kPagesCluster = 8;
constexpr int64_t kPagesInCluster = 2 * kPagesCluster * kPagesTokens;

cudaError_t pages_launch(PagesParams& p, int sm_count, cudaStream_t s)
{
    const size_t smem = pages_smem_bytes(p.B);
    p.state = p.total <= kPagesInCluster;
    if (p.state) {
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = kPagesCluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kPagesCluster);
        cfg.blockDim = dim3(kPagesThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, pages_update_kernel, p);
    }
    const int64_t ctas = std::min<int64_t>((p.total + kPagesTokens - 1) / kPagesTokens, 2 * sm_count);
    const cudaError_t e = launch_after(pages_update_kernel, dim3(unsigned(ctas)), kPagesThreads, smem, s, p);
    if (e != cudaSuccess) return e;
    return launch_after(pages_state_kernel, dim3(1), 1024, 0, s, p);
}

// What a call that needs more shared memory than a kernel gets unasked sets up once for each device (calls at the same
// time perhaps once each).
bool pages_smem(PagedDevice& st)
{
    if (st.wide_pages.load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(pages_update_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(pages_smem_bytes(kPagesMaxRows))) != cudaSuccess)
        return false;
    st.wide_pages.store(true, std::memory_order_release);
    return true;
}

template <class X, int kDim, bool kE4m3, bool kInterleaved, bool kSmallEps = false>
cudaError_t rotate_launch(NormRotateParams& p, bool vec, int sm_count, cudaStream_t s)
{
    // As many heads to a group of lanes as there is room for, shared out evenly, since their factors are made once;
    // fewer where that leaves SMs without work.
    constexpr int kGroups = kRotateThreads / (kDim / 8);
    const int64_t most = std::max(p.heads[0], p.heads[1]);  // (up to 2^31 - 1)
    const int64_t parts = (most + kRotateHeads<X> - 1) / kRotateHeads<X>;
    auto units = [&](int i) { return (int64_t(p.heads[i]) + p.per_unit - 1) / p.per_unit; };
    auto all_units = [&] { return units(0) + units(1); };
    for (p.per_unit = int32_t((most + parts - 1) / parts); p.per_unit > 1 && p.T * all_units() < int64_t(kGroups) * 2 * sm_count;)
        p.per_unit = (p.per_unit + 1) / 2;
    for (int i = 0; i < 2; ++i) p.units[i] = int32_t(units(i));
    p.by_units = FastDiv(uint32_t(all_units()));
    const size_t smem = size_t(rotate_smem<X>(p.per_unit));
    const dim3 grid(unsigned((p.T * all_units() + kGroups - 1) / kGroups));
    return vec ? launch_after(norm_rotate_kernel<X, kDim, kE4m3, true, kInterleaved, kSmallEps>, grid, kRotateThreads, smem, s, p)
               : launch_after(norm_rotate_kernel<X, kDim, kE4m3, false, kInterleaved, kSmallEps>, grid, kRotateThreads, smem, s, p);
}

template <class X, int kDim, bool kInterleaved>
cudaError_t rotate_to(NormRotateParams& p, bool e4m3, bool vec, int sm_count, cudaStream_t s)
{
    if (!e4m3) return rotate_launch<X, kDim, false, kInterleaved>(p, vec, sm_count, s);
    return p.eps >= kRotateEps ? rotate_launch<X, kDim, true, kInterleaved>(p, vec, sm_count, s)
                               : rotate_launch<X, kDim, true, kInterleaved, true>(p, vec, sm_count, s);
}

template <class X, int kDim>
cudaError_t rotate_dim(NormRotateParams& p, bool interleaved, bool e4m3, bool vec, int sm_count, cudaStream_t s)
{
    return interleaved ? rotate_to<X, kDim, true>(p, e4m3, vec, sm_count, s)
                       : rotate_to<X, kDim, false>(p, e4m3, vec, sm_count, s);
}

template <class X>
cudaError_t rotate_type(NormRotateParams& p, int32_t dim, bool interleaved, bool e4m3, bool vec, int sm_count, cudaStream_t s)
{
    return dim == 64 ? rotate_dim<X, 64>(p, interleaved, e4m3, vec, sm_count, s)
                     : rotate_dim<X, 128>(p, interleaved, e4m3, vec, sm_count, s);
}

int check_heads(const fp8mqa_heads* h, int32_t x_type, int32_t out_type)
{
    if (h->heads == 0) return FP8MQA_OK;
    if (!h->x || !h->out || (out_type == FP8MQA_E4M3) != (h->out_scale != nullptr)) return FP8MQA_ERR_INVALID_ARG;
    if (h->weight && h->weight_type != x_type && h->weight_type != FP8MQA_F32) return FP8MQA_ERR_INVALID_ARG;
    const uintptr_t e = uintptr_t(size_of(x_type));
    if (!on(h->x, e) || !on(h->out_scale, 4) || (h->weight && !on(h->weight, uintptr_t(size_of(h->weight_type)))))
        return FP8MQA_ERR_MISALIGNED;
    if (out_type != FP8MQA_E4M3) return on(h->out, e) ? FP8MQA_OK : FP8MQA_ERR_MISALIGNED;
    // E4M3 goes four values at a time
    return on(h->out, 4) && h->out_row_stride % 4 == 0 && h->out_head_stride % 4 == 0 ? FP8MQA_OK : FP8MQA_ERR_MISALIGNED;
}

// Whether each result lies apart from itself and from everything else, but for one that takes the place of its own rows:
// those are read by the lanes that write it, before they do.
bool results_apart(const fp8mqa_heads* const (&h)[2], int64_t T, int32_t dim, int64_t e, int64_t eo, const Places& positions,
                   const Places& inv_freq)
{
    Ascending read[6] = {positions, inv_freq}, written[4];  // then rows and a weight of each; results and scales
    bool in_place[2] = {false, false};
    int n = 0;
    for (; n < 2 && h[n]; ++n) {
        const fp8mqa_heads& t = *h[n];
        const Places x = {t.x, T, t.row_stride * e, t.heads, t.head_stride * e, dim * e};
        const Places out = {t.out, T, t.out_row_stride * eo, t.heads, t.out_head_stride * eo, dim * eo};
        if (!apart(out)) return false;
        in_place[n] = e == eo && same_places(x, out);
        read[2 + 2 * n] = x;
        read[3 + 2 * n] = bytes_at(t.weight, t.heads > 0 ? dim * size_of(t.weight_type) : 0);
        written[2 * n] = out;
        written[2 * n + 1] = bytes_at(t.out_scale, 4 * T * t.heads);
    }
    for (int i = 0; i < 2 * n; ++i) {
        for (int j = 0; j < 2 + 2 * n; ++j)
            if (meet(written[i], read[j]) && !(j == i + 2 && i % 2 == 0 && in_place[i / 2])) return false;
        for (int j = 0; j < i; ++j)
            if (meet(written[i], written[j])) return false;
    }
    return true;
}

}  // namespace
}  // namespace fp8mqa

extern "C" {

int fp8_mqa_pages_update(int32_t* table, int64_t table_stride, int32_t table_cols, int32_t page_size, int32_t* lens,
                         const int32_t* change, int64_t B, int32_t* free_pages, int64_t capacity, int32_t* n_free,
                         int64_t total, int32_t* slots, int32_t* positions, int32_t* rows, int32_t* starts,
                         int32_t* changed, void* stream)
{
    using namespace fp8mqa;
    if (B < 0 || table_cols < 0 || page_size < 1 || capacity < 0 || total < 0) return FP8MQA_ERR_INVALID_ARG;
    if (B > kPagesMaxRows || int64_t(table_cols) * page_size > INT32_MAX || B * table_cols > INT32_MAX || capacity > INT32_MAX || total > INT32_MAX)
        return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if ((B > 0 && (!lens || !change || !changed)) || (B > 0 && table_cols > 0 && !table) || (capacity > 0 && !free_pages) ||
        !n_free || !starts || (total > 0 && (!slots || !positions || !rows)))
        return FP8MQA_ERR_INVALID_ARG;
    // rows are written: they may not share memory
    if (B > 1 && table_stride < table_cols) return FP8MQA_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(table), static_cast<const void*>(lens), static_cast<const void*>(change),
                          static_cast<const void*>(free_pages), static_cast<const void*>(n_free),
                          static_cast<const void*>(slots), static_cast<const void*>(positions),
                          static_cast<const void*>(rows), static_cast<const void*>(starts),
                          static_cast<const void*>(changed)})
        if (!on(p, 4)) return FP8MQA_ERR_MISALIGNED;
    // what is written lies apart from everything else (`change` alone is not)
    const Ascending arrays[10] = {bytes_at(change, 4 * B),
                                  Places{table, B, 4 * table_stride, 1, 0, 4 * int64_t(table_cols)},
                                  bytes_at(lens, 4 * B),
                                  bytes_at(free_pages, 4 * capacity),
                                  bytes_at(n_free, 4),
                                  bytes_at(slots, 4 * total),
                                  bytes_at(positions, 4 * total),
                                  bytes_at(rows, 4 * total),
                                  bytes_at(starts, 4 * (B + 1)),
                                  bytes_at(changed, 4 * B)};
    for (int i = 1; i < 10; ++i)
        for (int j = 0; j < i; ++j)
            if (meet(arrays[i], arrays[j])) return FP8MQA_ERR_INVALID_ARG;
    int err = FP8MQA_OK;
    PagedDevice* st = paged_device(&err);
    if (!st) return err;
    // (what a kernel gets unasked is 48 KB)
    if (pages_smem_bytes(int32_t(B)) > 47 * 1024 && !pages_smem(*st)) return launched(cudaErrorInvalidValue);
    PagesParams p;
    p.table = table;
    p.table_stride = table_stride;
    p.cols = table_cols;
    p.page_size = page_size;
    p.by_page = FastDiv(uint32_t(page_size));
    p.lens = lens;
    p.change = change;
    p.B = int32_t(B);
    p.free_pages = free_pages;
    p.capacity = int32_t(capacity);
    p.n_free = n_free;
    p.total = int32_t(total);
    p.slots = slots;
    p.positions = positions;
    p.rows = rows;
    p.starts = starts;
    p.changed = changed;
    p.aligned = on(slots, 16) && on(positions, 16) && on(rows, 16);
    p.bounds = bounds_for(*st);
    spans(p.bounds, kMemTable, table, extent(B, 4 * table_stride, table_cols, 4, 1, 0, 4));
    spans(p.bounds, kMemLens, lens, 4 * B);
    spans(p.bounds, kMemIndices, change, 4 * B);
    spans(p.bounds, kMemFree, free_pages, 4 * capacity);
    spans(p.bounds, kMemFreeCount, n_free, 4);
    spans(p.bounds, kMemSlots, slots, 4 * total);
    spans(p.bounds, kMemPositions, positions, 4 * total);
    spans(p.bounds, kMemRows, rows, 4 * total);
    spans(p.bounds, kMemStarts, starts, 4 * (B + 1));
    spans(p.bounds, kMemOut, changed, 4 * B);
    return launched(pages_launch(p, st->sm_count, static_cast<cudaStream_t>(stream)));
}

int fp8_mqa_norm_rotate(const fp8mqa_heads* q, const fp8mqa_heads* k, int32_t x_type, int32_t out_type, int64_t T,
                        int32_t dim, const void* positions, int32_t position_bytes, const float* inv_freq,
                        int32_t rotated, int32_t interleaved, float eps, void* stream)
{
    using namespace fp8mqa;
    if (T < 0 || rotated < 0 || (interleaved != 0 && interleaved != 1) || (position_bytes != 4 && position_bytes != 8))
        return FP8MQA_ERR_INVALID_ARG;
    if ((x_type != FP8MQA_BF16 && x_type != FP8MQA_F16 && x_type != FP8MQA_F32) ||
        (out_type != x_type && out_type != FP8MQA_E4M3))
        return FP8MQA_ERR_INVALID_ARG;
    if ((dim != 64 && dim != 128) || rotated > dim || rotated % 16 != 0) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (!q || q->heads < 0 || (k && k->heads < 0)) return FP8MQA_ERR_INVALID_ARG;
    if (T == 0) return FP8MQA_OK;  // (empty tensors have no memory)
    int rc = check_heads(q, x_type, out_type);
    if (rc == FP8MQA_OK && k) rc = check_heads(k, x_type, out_type);
    if (rc != FP8MQA_OK) return rc;
    const int64_t heads = int64_t(q->heads) + (k ? k->heads : 0);
    if (T >= int64_t(1) << 31 || T * heads >= int64_t(1) << 31) return FP8MQA_ERR_UNSUPPORTED_SHAPE;
    if (heads == 0) return FP8MQA_OK;
    if (rotated > 0 && (!positions || !inv_freq)) return FP8MQA_ERR_INVALID_ARG;
    if (!on(positions, uintptr_t(position_bytes)) || !on(inv_freq, 4)) return FP8MQA_ERR_MISALIGNED;
    if (!results_apart({q, k}, T, dim, size_of(x_type), size_of(out_type), bytes_at(positions, rotated > 0 ? T * position_bytes : 0),
                       bytes_at(inv_freq, 2 * int64_t(rotated))))
        return FP8MQA_ERR_INVALID_ARG;
    int err = FP8MQA_OK;
    const PagedDevice* st = paged_device(&err);
    if (!st) return err;
    NormRotateParams p = {};
    p.bounds = bounds_for(*st);
    const int64_t e = size_of(x_type), eo = size_of(out_type);
    bool vec = true;
    for (int i = 0; i < 2; ++i) {
        const fp8mqa_heads* const h = i ? k : q;
        if (!h || h->heads == 0) continue;
        p.x[i] = h->x;
        p.row_stride[i] = h->row_stride;
        p.head_stride[i] = h->head_stride;
        p.weight[i] = h->weight;
        p.weight_f32[i] = h->weight_type == FP8MQA_F32;
        p.out[i] = h->out;
        p.out_row_stride[i] = h->out_row_stride;
        p.out_head_stride[i] = h->out_head_stride;
        p.out_scale[i] = h->out_scale;
        p.heads[i] = h->heads;
        // strides of dimensions of one are never used
        auto lies = [&](const void* at, int64_t row, int64_t head, int64_t size, uintptr_t bytes) {
            return on(at, bytes) && (T == 1 || row * size % int64_t(bytes) == 0) &&
                   (h->heads == 1 || head * size % int64_t(bytes) == 0);
        };
        vec = vec && on(h->weight, 16) && lies(h->x, h->row_stride, h->head_stride, e, 16) &&
              lies(h->out, h->out_row_stride, h->out_head_stride, eo, out_type == FP8MQA_E4M3 ? 8 : 16);
        spans(p.bounds, kMemRows + i, h->x, extent(T, h->row_stride * e, h->heads, h->head_stride * e, 1, 0, dim * e));
        spans(p.bounds, i ? kMemOut2 : kMemOut, h->out,
              extent(T, h->out_row_stride * eo, h->heads, h->out_head_stride * eo, 1, 0, dim * eo));
        spans(p.bounds, i ? kMemOutScale2 : kMemOutScale, h->out_scale, 4 * T * h->heads);
        spans(p.bounds, kMemWeight + i, h->weight, dim * size_of(h->weight_type));
    }
    p.T = int32_t(T);
    p.positions = positions;
    p.wide_positions = position_bytes == 8;
    p.inv_freq = inv_freq;
    p.rotated = rotated;
    p.eps = eps;
    spans(p.bounds, kMemPositions, positions, rotated > 0 ? T * position_bytes : 0);
    spans(p.bounds, kMemFreq, inv_freq, 4 * int64_t(rotated / 2));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool e4m3 = out_type == FP8MQA_E4M3;
    return launched(x_type == FP8MQA_BF16  ? rotate_type<__nv_bfloat16>(p, dim, interleaved, e4m3, vec, st->sm_count, s)
                    : x_type == FP8MQA_F16 ? rotate_type<__half>(p, dim, interleaved, e4m3, vec, st->sm_count, s)
                                           : rotate_type<float>(p, dim, interleaved, e4m3, vec, st->sm_count, s));
}

}  // extern "C"
