// Page tables, lengths, slots and positions of a step, from what each request's length changes by.
//
// With P the page size, request b of length n holds pages 0 .. ceil(n / P) - 1 of its table row.  The
// pages that nobody holds are a stack.  Shrinking requests give pages back, which go on the stack in the
// order of requests and columns; then growing requests take theirs off its top in the same order.  Three
// running sums over the requests say everything: new tokens, pages taken, pages given back.  The k-th page
// taken is the stack's k-th from the top, and a page above the stack's old top is one that this call gives
// back, which is read from where it lies in its request's row.  So nothing here waits for something that
// is written here: entries of the stack below its old top are only read, those above only written, rows
// that are read shrink and rows that are written grow.  Only the lengths and the stack's height are read
// by all and written, and those writes wait for everybody.
//
// The requests are few (8192 at most), so each CTA makes the running sums by itself, in shared memory, and
// the tokens, pages and requests are shared out to all threads of one cluster, whose barrier is what the
// writes of the lengths wait for: no workspace, no second kernel, no atomics.
#pragma once

#include "paged_common.cuh"

namespace fp8mqa {

constexpr int kPagesThreads = 1024;
constexpr int kPagesMaxRows = 8192;  // requests

struct PagesParams {
    int32_t* table;
    int64_t table_stride;
    int32_t cols, page_size;
    FastDiv by_page;
    int32_t* lens;
    const int32_t* change;
    int32_t B;
    int32_t* free_pages;
    int32_t capacity;
    int32_t* n_free;
    int32_t total;
    int32_t *slots, *positions, *rows, *starts, *changed;
    PagedBounds bounds;
};

// The last i in [0, n] with sums[i] <= x, of ascending sums with sums[0] <= x.
__device__ __forceinline__ int32_t last_at_most(const int32_t* sums, int32_t n, int32_t x)
{
    int32_t lo = 0, hi = n;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (sums[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// What a request is, and what it would be.
struct PagesRow {
    int32_t len, have;  // tokens and pages now
    int64_t to;         // tokens
    int32_t need;       // pages then
    bool fits;
    __device__ __forceinline__ PagesRow(const PagesParams& p, int32_t b)
    {
        const int32_t room = p.cols * p.page_size;  // under 2^31
        const int32_t n = in_bounds(p.bounds, kMemLens, p.lens + b, 4) ? p.lens[b] : 0;
        const int32_t d = in_bounds(p.bounds, kMemIndices, p.change + b, 4) ? p.change[b] : 0;
        len = min(max(n, 0), room);
        to = max(int64_t(0), int64_t(len) + d);
        fits = to <= room;
        have = pages(p, len);
        need = fits ? pages(p, int32_t(to)) : have;
    }
    __device__ __forceinline__ static int32_t pages(const PagesParams& p, int32_t n)
    {
        return n > 0 ? p.by_page.of(n - 1) + 1 : 0;
    }
};

__global__ void __launch_bounds__(kPagesThreads) pages_update_kernel(const __grid_constant__ PagesParams p)
{
    extern __shared__ int32_t s_sums[];  // running sums, B + 1 each: tokens, pages taken, pages given back
    __shared__ int64_t s_warp[3][kPagesThreads / 32];
    int32_t *const s_tokens = s_sums, *const s_taken = s_sums + (p.B + 1), *const s_given = s_taken + (p.B + 1);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- running sums, in 64 bits, kept up to 2^31 - 1: each thread counts some consecutive requests
    const int32_t per = (p.B + kPagesThreads - 1) / kPagesThreads;
    const int32_t b0 = min(per * tid, p.B), b1 = min(b0 + per, p.B);
    int64_t sum[3] = {0, 0, 0};
    auto add = [&](int32_t b) {
        const PagesRow r(p, b);
        sum[0] += max(int64_t(0), r.to - r.len);
        sum[1] += max(0, r.need - r.have);
        sum[2] += max(0, r.have - r.need);
    };
    for (int32_t b = b0; b < b1; ++b) add(b);
    int64_t mine[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        mine[i] = sum[i];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t x = __shfl_up_sync(~0u, sum[i], o);
            if (lane >= o) sum[i] += x;
        }
        if (lane == 31) s_warp[i][warp] = sum[i];
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            int64_t x = s_warp[i][lane];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            s_warp[i][lane] = x;
        }
    }
    __syncthreads();
    if (tid == 0) s_tokens[0] = s_taken[0] = s_given[0] = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) sum[i] += (warp ? s_warp[i][warp - 1] : 0) - mine[i];
    for (int32_t b = b0; b < b1; ++b) {
        add(b);
        s_tokens[b + 1] = int32_t(min(sum[0], int64_t(INT32_MAX)));
        s_taken[b + 1] = int32_t(min(sum[1], int64_t(INT32_MAX)));
        s_given[b + 1] = int32_t(min(sum[2], int64_t(INT32_MAX)));
    }
    __syncthreads();

    // ---- the stack: its height, then with what is given back, and what is taken off again
    const int32_t n0 = in_bounds(p.bounds, kMemFreeCount, p.n_free, 4) ? min(max(*p.n_free, 0), p.capacity) : 0;
    const int32_t n1 = n0 + min(s_given[p.B], p.capacity - n0);
    // requests that want pages get them up to the first one that the stack is too short for
    const int32_t taken = s_taken[last_at_most(s_taken, p.B, n1)];
    auto granted = [&](int32_t b, const PagesRow& r) { return r.fits && (r.need <= r.have || s_taken[b + 1] <= n1); };
    auto entry = [&](int32_t b, int32_t col) {
        const int32_t* const at = p.table + b * p.table_stride + col;
        return in_bounds(p.bounds, kMemTable, at, 4) ? *at : -1;
    };
    auto given = [&](int32_t i) {  // page number i of those given back
        const int32_t b = last_at_most(s_given, p.B, i);
        return entry(b, PagesRow(p, b).need + i - s_given[b]);
    };
    auto page_taken = [&](int32_t k) {
        const int32_t i = n1 - 1 - k;
        if (i >= n0) return given(i - n0);
        return in_bounds(p.bounds, kMemFree, p.free_pages + i, 4) ? p.free_pages[i] : -1;
    };
    auto put = [&](int kind, int32_t* to, int32_t x) {
        if (in_bounds(p.bounds, kind, to, 4)) *to = x;
    };

    const int32_t first = int32_t(blockIdx.x) * kPagesThreads + tid, step = int32_t(gridDim.x) * kPagesThreads;
    // ---- new tokens (counted in 64 bits: total may be close to 2^31)
    for (int64_t i = first; i < p.total; i += step) {
        int32_t slot = -1, position = 0, b = 0;
        if (i < s_tokens[p.B]) {
            b = last_at_most(s_tokens, p.B, int32_t(i));
            const PagesRow r(p, b);
            const int64_t at = int64_t(r.len) + int32_t(i) - s_tokens[b];
            position = int32_t(min(at, int64_t(INT32_MAX)));
            if (granted(b, r)) {
                const int32_t col = p.by_page.of(position);
                const int32_t page = col < r.have ? entry(b, col) : page_taken(s_taken[b] + col - r.have);
                const int64_t x = int64_t(page) * p.page_size + (position - col * p.page_size);
                if (page >= 0 && x <= INT32_MAX) slot = int32_t(x);
            }
        }
        put(kMemSlots, p.slots + i, slot);
        put(kMemPositions, p.positions + i, position);
        put(kMemRows, p.rows + i, b);
    }
    // ---- pages taken go into their rows, pages given back and left over on the stack
    for (int64_t k = first; k < taken; k += step) {
        const int32_t b = last_at_most(s_taken, p.B, int32_t(k));
        put(kMemTable, p.table + b * p.table_stride + PagesRow(p, b).have + (int32_t(k) - s_taken[b]), page_taken(int32_t(k)));
    }
    for (int64_t i = int64_t(n0) + first; i < n1 - taken; i += step)
        put(kMemFree, p.free_pages + i, given(int32_t(i) - n0));
    // ---- requests
    for (int32_t b = first; b <= p.B; b += step) {
        put(kMemStarts, p.starts + b, s_tokens[b]);
        if (b == p.B) break;
        const PagesRow r(p, b);
        put(kMemOut, p.changed + b, granted(b, r) ? int32_t(r.to) - r.len : 0);
    }
    // ---- nobody reads the lengths and the stack's height any more
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int32_t b = first; b < p.B; b += step) {
        const PagesRow r(p, b);
        put(kMemLens, p.lens + b, granted(b, r) ? int32_t(r.to) : r.len);
    }
    if (first == 0) put(kMemFreeCount, p.n_free, n1 - taken);
}

}  // namespace fp8mqa
