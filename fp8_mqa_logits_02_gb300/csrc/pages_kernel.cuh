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
// the tokens, pages and requests are shared out to all threads: no workspace, no atomics.  A thread finds four
// tokens side by side with one search and one page, or two.  A call is one cluster, whose barrier the lengths
// and the height wait for (everyone arrives there early, after the sums); a large one is as many CTAs as its
// tokens want, and then a small kernel for the lengths and the height.
//
// Measured: 256 requests that stay as they are 3.4 us, with two new tokens each 6.5; 256 requests of which 16 end (165
// thousand tokens) and 240 grow (by 3 thousand), and then the reverse, 17 us for both calls (41 with a search, two loads
// and three stores a token); 64 requests and 27 thousand tokens 8.7 us a call.  The chain of dependent loads and searches
// decides, not the bytes (2 MB, 0.3 us).
#pragma once

#include "paged_common.cuh"

namespace fp8mqa {

constexpr int kPagesThreads = 256;
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
    int32_t aligned;  // slots, positions and rows lie on 16 bytes
    int32_t state;    // whether the lengths and the stack's height are written too
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
    // running sums, B + 1 each: tokens, pages taken, pages given back; and the lengths (~n of requests that do not fit)
    extern __shared__ int32_t s_sums[];
    __shared__ uint32_t s_warp[3][kPagesThreads / 32];
    int32_t *const s_tokens = s_sums, *const s_taken = s_sums + (p.B + 1), *const s_given = s_taken + (p.B + 1);
    int32_t* const s_len = s_given + (p.B + 1);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- what each request wants, and running sums of it: each thread takes some consecutive requests.  Pages are
    // under 2^31 in all; tokens may be more, and their sums stop there
    const int32_t n_free = in_bounds(p.bounds, kMemFreeCount, p.n_free, 4) ? *p.n_free : 0;
    const int32_t per = (p.B + kPagesThreads - 1) / kPagesThreads;
    const int32_t b0 = min(per * tid, p.B), b1 = min(b0 + per, p.B);
    uint32_t sum[3] = {0, 0, 0};
    auto add = [](uint32_t a, uint32_t b) { return min(a + b, uint32_t(INT32_MAX)); };  // of numbers up to that
    for (int32_t b = b0; b < b1; ++b) {
        const PagesRow r(p, b);
        s_len[b] = r.fits ? r.len : ~r.len;
        s_tokens[b + 1] = int32_t(min(max(int64_t(0), r.to - r.len), int64_t(INT32_MAX)));
        s_taken[b + 1] = max(0, r.need - r.have);
        s_given[b + 1] = max(0, r.have - r.need);
        sum[0] = add(sum[0], s_tokens[b + 1]);
        sum[1] += s_taken[b + 1];
        sum[2] += s_given[b + 1];
    }
    uint32_t before[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint32_t x = sum[i];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x = add(x, y);
        }
        if (lane == 31) s_warp[i][warp] = x;
        before[i] = __shfl_up_sync(~0u, x, 1);
        if (lane == 0) before[i] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w)
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (w < warp) before[i] = add(before[i], s_warp[i][w]);
    if (tid == 0) s_tokens[0] = s_taken[0] = s_given[0] = 0;
    for (int32_t b = b0; b < b1; ++b) {
        s_tokens[b + 1] = before[0] = add(before[0], s_tokens[b + 1]);
        s_taken[b + 1] = before[1] += s_taken[b + 1];
        s_given[b + 1] = before[2] += s_given[b + 1];
    }
    __syncthreads();

    // ---- the stack: its height, then with what is given back, and what is taken off again.  Requests that want pages
    // get them up to the first one that it is too short for
    const int32_t n0 = min(max(n_free, 0), p.capacity);
    const int32_t n1 = n0 + min(s_given[p.B], p.capacity - n0);
    const int32_t taken = s_taken[last_at_most(s_taken, p.B, n1)];
    for (int32_t b = b0; b < b1; ++b)
        if (s_len[b] >= 0 && s_taken[b + 1] > s_taken[b] && s_taken[b + 1] > n1) s_len[b] = ~s_len[b];
    __syncthreads();
    if (p.state) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // all of them has been read
    auto length = [&](int32_t b) { return s_len[b] < 0 ? ~s_len[b] : s_len[b]; };
    auto have = [&](int32_t b) { return PagesRow::pages(p, length(b)); };
    auto entry = [&](int32_t b, int32_t col) {
        const int32_t* const at = p.table + b * p.table_stride + col;
        return in_bounds(p.bounds, kMemTable, at, 4) ? *at : -1;
    };
    auto given = [&](int32_t i) {  // page number i of those given back
        const int32_t b = last_at_most(s_given, p.B, i);
        return entry(b, have(b) - s_given[b + 1] + i);
    };
    auto page_taken = [&](int32_t k) {
        const int32_t i = n1 - 1 - k;
        if (i >= n0) return given(i - n0);
        return in_bounds(p.bounds, kMemFree, p.free_pages + i, 4) ? p.free_pages[i] : -1;
    };
    auto page_of = [&](int32_t b, int32_t col) {  // of a request that fits, then
        const int32_t held = have(b);
        return col < held ? entry(b, col) : page_taken(s_taken[b] + col - held);
    };
    auto slot_of = [&](int32_t page, int32_t in_page) {
        const int64_t x = int64_t(page) * p.page_size + in_page;
        return page >= 0 && x <= INT32_MAX ? int32_t(x) : -1;
    };
    auto put = [&](int kind, int32_t* to, int32_t x) {
        if (in_bounds(p.bounds, kind, to, 4)) *to = x;
    };

    // (each kind of work begins with CTAs of its own, so that in a small call nothing waits for another kind)
    const int32_t step = int32_t(gridDim.x) * kPagesThreads;
    auto place = [&](unsigned from) {
        return int32_t((blockIdx.x + gridDim.x - from % gridDim.x) % gridDim.x) * kPagesThreads + tid;
    };
    const int32_t first = place(0), first_taken = place(5), first_given = place(6);
    // ---- new tokens, four side by side a thread (counted in 64 bits: total may be close to 2^31)
    const int32_t all = s_tokens[p.B];
    for (int64_t i0 = 4 * int64_t(first); i0 < p.total; i0 += 4 * int64_t(step)) {
        alignas(16) int32_t slot[4], position[4], row[4];
        const int32_t i = int32_t(i0), b = i0 < all ? last_at_most(s_tokens, p.B, i) : 0;
        const int32_t at = i0 < all ? s_len[b] + (i - s_tokens[b]) : 0;  // (one that does not fit: below 0, or not looked at)
        const int32_t col = p.by_page.of(max(at, 0)), in_page = at - col * p.page_size;
        if (i0 + 4 <= all && i0 + 4 <= s_tokens[b + 1] && s_len[b] >= 0 && p.page_size >= 4) {
            // of one request, on one page or two
            const int32_t page = page_of(b, col), left = p.page_size - in_page;  // tokens on the first page
            const int32_t next = left < 4 ? page_of(b, col + 1) : page;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                slot[k] = k < left ? slot_of(page, in_page + k) : slot_of(next, k - left);
                position[k] = at + k;
                row[k] = b;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                int32_t s = -1, n = 0, r = 0;
                if (i0 + k < all && i0 + k < p.total) {
                    r = last_at_most(s_tokens, p.B, i + k);
                    n = int32_t(min(int64_t(length(r)) + (i + k - s_tokens[r]), int64_t(INT32_MAX)));
                    if (s_len[r] >= 0) {
                        const int32_t c = p.by_page.of(n);
                        s = slot_of(page_of(r, c), n - c * p.page_size);
                    }
                }
                slot[k] = s;
                position[k] = n;
                row[k] = r;
            }
        }
        if (p.aligned && i0 + 4 <= p.total && in_bounds(p.bounds, kMemSlots, p.slots + i0, 16) &&
            in_bounds(p.bounds, kMemPositions, p.positions + i0, 16) && in_bounds(p.bounds, kMemRows, p.rows + i0, 16)) {
            *reinterpret_cast<int4*>(p.slots + i0) = *reinterpret_cast<const int4*>(slot);
            *reinterpret_cast<int4*>(p.positions + i0) = *reinterpret_cast<const int4*>(position);
            *reinterpret_cast<int4*>(p.rows + i0) = *reinterpret_cast<const int4*>(row);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k < p.total) {
                    put(kMemSlots, p.slots + i0 + k, slot[k]);
                    put(kMemPositions, p.positions + i0 + k, position[k]);
                    put(kMemRows, p.rows + i0 + k, row[k]);
                }
        }
    }
    // ---- pages taken go into their rows, pages given back and left over on the stack; a few at a time, whose loads
    // hang on nothing of one another
    constexpr int kBatch = 4;
    for (int64_t k0 = first_taken; k0 < taken; k0 += kBatch * int64_t(step)) {
        int32_t page[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            page[j] = k0 + j * int64_t(step) < taken ? page_taken(int32_t(k0 + j * int64_t(step))) : 0;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t k = k0 + j * int64_t(step);
            if (k >= taken) break;
            const int32_t b = last_at_most(s_taken, p.B, int32_t(k));
            put(kMemTable, p.table + b * p.table_stride + have(b) + (int32_t(k) - s_taken[b]), page[j]);
        }
    }
    const int32_t left = n1 - taken - n0;  // of those given back
    for (int64_t k0 = first_given; k0 < left; k0 += kBatch * int64_t(step)) {
        int32_t page[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            page[j] = k0 + j * int64_t(step) < left ? given(int32_t(k0 + j * int64_t(step))) : 0;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (k0 + j * int64_t(step) < left) put(kMemFree, p.free_pages + n0 + k0 + j * int64_t(step), page[j]);
    }
    // ---- requests: the last CTA's, whose threads have theirs at hand
    if (blockIdx.x == gridDim.x - 1) {
        if (tid == 0) put(kMemStarts, p.starts, 0);
        for (int32_t b = b0; b < b1; ++b) {
            const PagesRow r(p, b);
            put(kMemStarts, p.starts + b + 1, s_tokens[b + 1]);
            put(kMemOut, p.changed + b, s_len[b] >= 0 ? int32_t(r.to) - r.len : 0);
        }
    }
    if (p.state) {
        __syncwarp();  // the lanes had different numbers of tokens and pages
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (blockIdx.x == gridDim.x - 1) {
            for (int32_t b = b0; b < b1; ++b) {
                const PagesRow r(p, b);
                put(kMemLens, p.lens + b, s_len[b] >= 0 ? int32_t(r.to) : r.len);
            }
            if (tid == 0) put(kMemFreeCount, p.n_free, n1 - taken);
        }
    }
}

// The lengths and the height after a launch that wrote the results: by the changes that it granted.
__global__ void __launch_bounds__(1024) pages_state_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ int32_t s_pages[2][32];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t n_free = in_bounds(p.bounds, kMemFreeCount, p.n_free, 4) ? *p.n_free : 0;
    const int32_t room = p.cols * p.page_size;
    int32_t taken = 0, given = 0;
    for (int32_t b = tid; b < p.B; b += 1024) {
        if (!in_bounds(p.bounds, kMemLens, p.lens + b, 4) || !in_bounds(p.bounds, kMemOut, p.changed + b, 4)) continue;
        const int32_t len = min(max(p.lens[b], 0), room), to = len + p.changed[b];
        const int32_t more = PagesRow::pages(p, to) - PagesRow::pages(p, len);
        taken += max(more, 0);
        given += max(-more, 0);
        p.lens[b] = to;
    }
    taken = int32_t(__reduce_add_sync(~0u, uint32_t(taken)));
    given = int32_t(__reduce_add_sync(~0u, uint32_t(given)));
    if (lane == 0) {
        s_pages[0][warp] = taken;
        s_pages[1][warp] = given;
    }
    __syncthreads();
    if (warp == 0) {
        taken = int32_t(__reduce_add_sync(~0u, uint32_t(s_pages[0][lane])));
        given = int32_t(__reduce_add_sync(~0u, uint32_t(s_pages[1][lane])));
        const int32_t n0 = min(max(n_free, 0), p.capacity);
        if (lane == 0 && in_bounds(p.bounds, kMemFreeCount, p.n_free, 4))
            *p.n_free = n0 + min(given, p.capacity - n0) - taken;
    }
}

}  // namespace fp8mqa
