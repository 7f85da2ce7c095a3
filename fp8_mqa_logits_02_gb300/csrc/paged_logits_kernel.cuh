// The indexer logits of each sequence's T newest tokens, read straight from the cache's pages:
//
//   out[b*T + t, n] = scale[n] * sum_h relu(q[b,t,h] . k[n]) * w[b,t,h],  n < len[b] - (T - 1 - t)
//
// Bound: a key is 132 bytes and gives T logits of 4, so the cache's bytes decide.  The products
// (8192 flops a key and token) go to tcgen05: at the rate at which HBM gives keys that is 415 TFLOP/s
// for one token, 1.7 PFLOP/s for four, more than the warps' own matrix instructions can be asked for.
//
// A CTA's four warps do everything, a tile of 128 keys at a time (thread = key = TMEM lane):
//   copy      each warp copies its 32 keys' rows into a ring of kStages tiles, as the 128-byte swizzle
//             of the MMA wants them, wherever their pages lie; two stages or three are in flight;
//   multiply  one thread issues S[key, (t, h)] = K Q^T for the tile whose copies are done, into one
//             of two TMEM buffers;
//   finish    meanwhile the threads take the previous tile's S: relu, times w, the sum over 32 heads
//             in registers, times the key's scale, a coalesced store.
//
// Split: the rows' tiles, and for clean_logits their -inf spans, are laid end to end by cost, and
// every CTA takes an equal share; it writes its -inf spans while its first copies are under way.
// A CTA's stream of tiles runs on from row to row; Q and w have kSlots slots for that.
//
// The waits for the tensor core are bounded (PagedLogitsParams::wait_ns); on expiry the CTA reports
// it in the status word, waits for its MMAs once more, frees its tensor memory and returns.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"
#include "sm103_ptx.cuh"

namespace fp8mqa {

struct PagedLogitsParams {
    const uint8_t* q;
    const float* w;
    PagedView keys;
    RowUnits units;
    PageTable table;
    const int32_t* lens;
    float* out;
    int64_t ld, N, B;
    int32_t T, clean;
    int32_t aligned;  // rows of out start on 16 bytes
    int32_t* status;
    uint64_t wait_ns;
};

constexpr int kPagedHeads = 32, kPagedDim = 128;
constexpr int kPagedThreads = 128, kPagedWarps = kPagedThreads / 32, kPagedTile = 128;
constexpr int kPagedMmaK = 32;     // E4M3 values of a tcgen05.mma
constexpr int kPagedFill = 1024;  // columns of a -inf span
constexpr int32_t kPagedTimeout = 1;           // status bit: a bounded wait gave up
constexpr uint64_t kPagedDrainNs = 1000000000ull;  // bound of the last wait before a CTA gives up

// kTok: tokens of a CTA (1, 2 or 4).
template <int kTok>
struct PagedShape {
    static constexpr int kStages = kTok == 2 ? 4 : 3;
    static constexpr int kSlots = 3;  // rows whose Q and w are held: of the tile being finished and two on
    static constexpr int kCtasPerSm = kTok == 1 ? 3 : 2;
    static constexpr uint32_t kN = kTok * kPagedHeads;
    static constexpr uint32_t kTmemCols = 2 * kN;
    static constexpr uint32_t kKBytes = kPagedTile * kPagedDim, kQBytes = kN * kPagedDim;
    static constexpr uint32_t kOffQ = kStages * kKBytes;
    static constexpr uint32_t kOffW = kOffQ + kSlots * kQBytes;
    static constexpr uint32_t kOffScale = kOffW + kSlots * kN * 4;
    static constexpr uint32_t kOffItem = kOffScale + kStages * kPagedTile * 4;
    static constexpr uint32_t kOffBar = kOffItem + kStages * 32;
    static constexpr uint32_t kSmem = kOffBar + 32 + 1024;  // slack for aligning the base
    // D f32, A = B = E4M3, both K-major, M = 128 keys
    static constexpr uint32_t kIdesc = (1u << 4) | ((kN >> 3) << 17) | (uint32_t(kPagedTile >> 4) << 24);
};

// A tile in the ring.
struct PagedItem {
    int64_t b;
    int32_t tile, row;   // row: the CTA's running number of its rows
    uint32_t there[4];   // which keys are there
};
static_assert(sizeof(PagedItem) == 32, "PagedShape::kOffItem");

__device__ __forceinline__ void tmem_ld_32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

template <int kTok>
__global__ void __launch_bounds__(kPagedThreads, PagedShape<kTok>::kCtasPerSm)
    paged_logits_kernel(const __grid_constant__ PagedLogitsParams p)
{
    using S = PagedShape<kTok>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t s_scan[kPagedWarps], s_first[2];
    __shared__ uint32_t s_tmem;
    uint8_t* const smem =
        smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int t0 = blockIdx.y * kTok, n_tok = min(kTok, p.T - t0);
    const int64_t cap = min(p.N, int64_t(p.table.cols) * p.keys.page_size);

    // ---- the rows' costs, in units of about half a kilobyte moved
    const int64_t c_tile = 34 + n_tok, c_fill = 8 * n_tok;
    auto length = [&](int64_t b) {
        const int64_t n = __ldg(p.lens + b);
        return int32_t(n < 0 ? 0 : n < cap ? n : cap);
    };
    auto tiles = [&](int64_t b) { return (length(b) + kPagedTile - 1) / kPagedTile; };
    auto fills = [&](int32_t n_tiles) {
        const int64_t left = p.N - int64_t(n_tiles) * kPagedTile;
        return !p.clean || left <= 0 ? int64_t(0) : (left + kPagedFill - 1) / kPagedFill;
    };
    auto cost = [&](int64_t b) {
        const int32_t n = tiles(b);
        return n * c_tile + fills(n) * c_fill;
    };
    const int64_t per = (p.B + kPagedThreads - 1) / kPagedThreads;
    const int64_t b1 = min(per * (tid + 1), p.B);
    int64_t sum = 0;
    for (int64_t b = per * tid; b < b1; ++b) sum += cost(b);
    int64_t scan = sum, total = 0, before = 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += x;
    }
    if (lane == 31) s_scan[warp] = scan;

    // ---- tensor memory and barriers
    const uint32_t bar = base + S::kOffBar;  // two: one for each TMEM buffer
    if (warp == 0) {
        // the permit is given up at once: while a CTA holds it, the SM's next CTA waits in its alloc
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), S::kTmemCols);
        ptx::tmem_relinquish();
    }
    if (tid == 0) {
        ptx::mbar_init(bar, 1);
        ptx::mbar_init(bar + 8, 1);
        ptx::mbar_init_fence();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_tmem;
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) {
        if (w == warp) before = total + scan - sum;
        total += s_scan[w];
    }
    const int64_t from = blockIdx.x * total / gridDim.x, to = (blockIdx.x + 1) * total / gridDim.x;
    if (before <= from && from < before + sum) {
        int64_t b = per * tid, at = before;
        for (;; ++b) {
            const int64_t c = cost(b);
            if (from < at + c) break;
            at += c;
        }
        s_first[0] = b;
        s_first[1] = at;
    }
    __syncthreads();

    // ---- the stream of this CTA's tiles: those whose cost begins in [from, to)
    int64_t next_b = s_first[0], next_at = s_first[1];  // the next row, the cost before it
    if (from >= to) next_at = to;
    int64_t cur_b = 0;
    int32_t cur_tile = 0, cur_end = 0, cur_len = 0, cur_row = -1;  // the row being copied
    auto more = [&] {  // whether there is a tile to copy; moves on to its row
        while (cur_tile >= cur_end) {
            if (next_at >= to) return false;
            cur_b = next_b++;
            cur_len = length(cur_b);
            const int32_t n = (cur_len + kPagedTile - 1) / kPagedTile;
            const int64_t lo = from > next_at ? (from - next_at + c_tile - 1) / c_tile : 0;
            const int64_t hi = (to - next_at + c_tile - 1) / c_tile;
            cur_tile = int32_t(min(lo, int64_t(n)));
            cur_end = int32_t(min(hi, int64_t(n)));
            next_at += n * c_tile + fills(n) * c_fill;
            cur_row = -1;  // not numbered yet
        }
        return true;
    };
    // ---- copies
    int32_t copied = 0, rows_copied = 0;
    auto copy = [&] {  // the tile that more() found, and its row's Q and w with the first one
        const int stage = copied % S::kStages;
        const int32_t n = cur_tile * kPagedTile + tid;
        int32_t page = -1, row = 0;
        const bool there = n < cur_len && locate(p.keys, p.table, cur_b, n, &page, &row);
        const uint32_t at = there ? page * p.units.page + row * p.units.row : kNoRow;
        const uint32_t dst = base + stage * S::kKBytes;
        const int c = lane % 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = j * 4 + lane / 8;
            const uint32_t from_row = __shfl_sync(~0u, at, r);
            const bool ok = from_row != kNoRow;
            copy16(dst + (warp * 32 + r) * 128 + 16 * (c ^ (r & 7)),
                   p.keys.data + uint64_t(ok ? from_row : 0) * p.units.unit + 16 * c, ok);
        }
        copy4(base + S::kOffScale + (stage * kPagedTile + tid) * 4,
              p.keys.scale + (there ? int64_t(page) * p.keys.scale_page_stride +
                                          int64_t(row) * p.keys.scale_row_stride
                                    : 0),
              there);
        const uint32_t here = __ballot_sync(~0u, there);
        if (cur_row < 0) {  // the row's first tile
            cur_row = rows_copied++;
            const int slot = cur_row % S::kSlots;
            const int64_t first = (cur_b * p.T + t0) * kPagedHeads;
            for (int i = tid; i < n_tok * kPagedHeads * 8; i += kPagedThreads)
                copy16(base + S::kOffQ + slot * S::kQBytes + i / 8 * 128 + 16 * (i % 8 ^ (i / 8 & 7)),
                       p.q + (first + i / 8) * kPagedDim + 16 * (i % 8), true);
            for (int i = tid; i < n_tok * kPagedHeads / 4; i += kPagedThreads)
                copy16(base + S::kOffW + slot * S::kN * 4 + 16 * i, p.w + first + 4 * i, true);
        }
        PagedItem* const item = reinterpret_cast<PagedItem*>(smem + S::kOffItem) + stage;
        if (lane == 0) item->there[warp] = here;
        if (tid == 0) {
            item->b = cur_b;
            item->tile = cur_tile;
            item->row = cur_row;
        }
        copy_commit();
        ++copied;
        ++cur_tile;
    };
    // Waits until tile i is multiplied, for `limit` ns at most.
    auto wait = [&](int32_t i, uint64_t limit) {
        const uint32_t at = bar + 8 * (i & 1), parity = uint32_t(i >> 1) & 1u;
        if (ptx::mbar_try_wait(at, parity)) return true;
        const uint64_t start = ptx::globaltimer_ns();
        while (!ptx::mbar_try_wait_sleep(at, parity, 20000))
            if (ptx::globaltimer_ns() - start > limit) return false;
        return true;
    };

    // ---- the first copies, and the -inf spans while they are under way
    int32_t row_done = 0;  // the number of the row whose tile was finished last (or comes first)
    auto allowed = [&] {   // whether the next tile's row has a slot
        return cur_row >= 0 || rows_copied - row_done < S::kSlots;
    };
    while (copied < S::kStages - 1 && more() && allowed()) copy();
    if (p.clean) {
        int64_t at = s_first[1];
        for (int64_t b = s_first[0]; at < to; ++b) {
            const int32_t n = tiles(b);
            const int64_t n_fill = fills(n), begin = at + n * c_tile;
            at = begin + n_fill * c_fill;
            const int64_t lo = from > begin ? (from - begin + c_fill - 1) / c_fill : 0;
            const int64_t hi = min(n_fill, (to - begin + c_fill - 1) / c_fill);
            for (int64_t f = lo; f < hi; ++f) {
                const int64_t c0 = int64_t(n) * kPagedTile + f * kPagedFill;
                const int64_t c1 = min(p.N, c0 + kPagedFill);
                for (int t = 0; t < n_tok; ++t) {
                    float* const out = p.out + (b * p.T + t0 + t) * p.ld;
                    if (p.aligned) {
                        const int64_t c4 = c0 + (c1 - c0) / 4 * 4;
                        for (int64_t c = c0 + 4 * tid; c < c4; c += 4 * kPagedThreads)
                            __stcs(reinterpret_cast<float4*>(out + c),
                                   make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F,
                                               -CUDART_INF_F));
                        if (c4 + tid < c1) __stcs(out + c4 + tid, -CUDART_INF_F);
                    } else {
                        for (int64_t c = c0 + tid; c < c1; c += kPagedThreads)
                            __stcs(out + c, -CUDART_INF_F);
                    }
                }
            }
        }
    }

    // ---- tile i multiplied while tile i - 1 is finished
    bool late = false;
    int32_t issued = 0;
    int64_t prev_b = 0;
    int32_t prev_tile = 0, prev_row = 0, prev_len = 0;
    uint32_t prev_there = 0;
    float prev_scale = 0.0f;
    for (int32_t i = 0;; ++i) {
        const bool any = i < copied;  // the same in all threads
        if (any) {
            const int behind = copied - 1 - i;  // copies after this tile's
            if (behind <= 0)
                copy_wait<0>();
            else if (behind == 1)
                copy_wait<1>();
            else
                copy_wait<2>();
            ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before();  // tile i - 2 is read from the buffer that tile i takes
        if (__syncthreads_or(late) || (!any && i == 0)) break;
        PagedItem item;
        uint32_t there = 0;
        float scale = 0.0f;
        int32_t len = 0;
        if (any) {
            const int stage = i % S::kStages;
            const PagedItem* const at = reinterpret_cast<const PagedItem*>(smem + S::kOffItem) + stage;
            item.b = at->b;
            item.tile = at->tile;
            item.row = at->row;
            there = at->there[warp];
            scale = reinterpret_cast<const float*>(smem + S::kOffScale)[stage * kPagedTile + tid];
            len = __ldg(p.lens + item.b);
            if (tid == 0) {
                ptx::tc_fence_after();
                const uint64_t a = sw128_desc(base + stage * S::kKBytes);
                const uint64_t q = sw128_desc(base + S::kOffQ + item.row % S::kSlots * S::kQBytes);
#pragma unroll
                for (int k = 0; k < kPagedDim / kPagedMmaK; ++k)
                    ptx::mma_f8f6f4(tmem + (i & 1) * S::kN, a + 2ull * k, q + 2ull * k, S::kIdesc,
                                    k > 0 ? 1u : 0u);
                ptx::mma_commit(bar + 8 * (i & 1));
            }
            __syncwarp();
            ++issued;
        }
        if (i > 0) {
            late = __any_sync(~0u, !wait(i - 1, p.wait_ns));
            row_done = prev_row;
        }
        // every MMA before tile i is done, so the stage of tile i - 1 is free
        while (!late && copied < i + S::kStages && more() && allowed()) copy();
        if (i > 0 && !late) {
            ptx::tc_fence_after();
            const float* const w =
                reinterpret_cast<const float*>(smem + S::kOffW) + prev_row % S::kSlots * S::kN;
            const int64_t n = int64_t(prev_tile) * kPagedTile + tid;
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                if (t >= n_tok) break;
                uint32_t x[kPagedHeads];
                tmem_ld_32(tmem + (uint32_t(warp * 32) << 16) + ((i - 1) & 1) * S::kN + t * kPagedHeads,
                           x);
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < kPagedHeads; h += 4) {
                    const float4 wh = *reinterpret_cast<const float4*>(w + t * kPagedHeads + h);
                    y[0] = fmaf(fmaxf(__uint_as_float(x[h]), 0.0f), wh.x, y[0]);
                    y[1] = fmaf(fmaxf(__uint_as_float(x[h + 1]), 0.0f), wh.y, y[1]);
                    y[2] = fmaf(fmaxf(__uint_as_float(x[h + 2]), 0.0f), wh.z, y[2]);
                    y[3] = fmaf(fmaxf(__uint_as_float(x[h + 3]), 0.0f), wh.w, y[3]);
                }
                const float sum = ((y[0] + y[1]) + (y[2] + y[3])) * prev_scale;
                const bool seen = n < min(int64_t(prev_len) - (p.T - 1 - (t0 + t)), cap);
                if (n < p.N && (seen || p.clean))
                    __stcs(p.out + (prev_b * p.T + t0 + t) * p.ld + n,
                           seen && (prev_there >> lane & 1u) ? sum : -CUDART_INF_F);
            }
        }
        if (!any) break;
        prev_b = item.b;
        prev_tile = item.tile;
        prev_row = item.row;
        prev_there = there;
        prev_scale = scale;
        prev_len = len;
    }

    // ---- the end; after a wait that gave up, the MMAs under way get kPagedDrainNs more
    copy_wait<0>();
    if (__syncthreads_or(late)) {
        if (tid == 0) {
            atomicOr(p.status, kPagedTimeout);
            if (issued > 0) wait(issued - 1, kPagedDrainNs);
        }
        __syncthreads();
    }
    if (warp == 0) ptx::tmem_dealloc(tmem, S::kTmemCols);
}

}  // namespace fp8mqa
