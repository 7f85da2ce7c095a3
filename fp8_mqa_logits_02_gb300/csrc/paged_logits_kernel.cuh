// The indexer logits of each sequence's T newest tokens, read straight from the cache's pages:
//
//   out[b*T + t, n] = scale[n] * sum_h relu(q[b,t,h] . k[n]) * w[b,t,h],  n < len[b] - (T - 1 - t)
//
// Bound: a key is 132 bytes and gives T logits of 4, so the cache's bytes decide.  The products
// (8192 flops a key and token) go to tcgen05: at the rate at which HBM gives keys that is 415 TFLOP/s
// for one token, 1.7 PFLOP/s for four, more than the warps' own matrix instructions can be asked for.
//
// Warps of a CTA, a tile of 128 keys at a time (thread = key = TMEM lane):
//   copy         fills a ring of kStages tiles, as the 128-byte swizzle of the MMA wants them, wherever
//                their pages lie.  kTma: one warp, a lane for each page's piece of the tile (boxes of
//                a power of two of rows that divides the page); else four warps by 16-byte
//                asynchronous copies, their keys' pages looked up a tile ahead;
//   multiply (1) one thread issues S[key, (t, h)] = K Q^T into one of two TMEM buffers;
//   finish (8)   S from TMEM, relu, times w, the sum over 32 heads in registers, times the key's scale,
//                a coalesced store; four warps take the even tiles (and their buffer), four the odd ones;
//   fill (1)     clean_logits: the -inf spans.
// (With four warps doing it all in turn the chain of a tile's steps decided: 1.65 us a tile, 47 us for
// 64 rows x 2 tokens.)
//
// Measured: 64 rows of up to 32767 keys x 2 tokens (156 MB) 30.1 us, 5.2 TB/s, of which 4 us are start and
// tail; x 4 tokens 35.1 us; one row of 131072 keys 7.0 us with the keys in L2, 8.2 us from HBM; one of 4096
// 4.3 us.
//
// Split: the rows' tiles and -inf spans are laid end to end by cost, and every CTA takes an equal
// share.  A CTA's stream of tiles runs on from row to row; Q and w have kSlots slots for that.
//
// Every wait is bounded (PagedLogitsParams::wait_ns); on expiry the CTA reports it in the status
// word, all its warps stop, its MMAs under way get kPagedDrainNs more, and it frees its tensor memory.
#pragma once

#include <cuda.h>
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
    int32_t* status;
    uint64_t wait_ns;
    uint32_t suspend_ns;     // of one suspension within a wait, at most
    int32_t box, box_shift;  // kTma: rows of a piece, 2^box_shift
    uint32_t page_rows;      // kTma: rows of the tensor map from page to page
    PagedBounds bounds;
};

constexpr int kPagedHeads = 32, kPagedDim = 128;
constexpr int kPagedTile = 128;
constexpr int kPagedFinishWarps = 8, kPagedScanThreads = 128;
// Tiles that a copy warp leaves under way when it reports one (copies of 16 bytes; TMA reports by itself):
// with 2, 64 rows x 4 tokens (three stages) on pages of 16 take 58.1 us instead of 46.1, one or two tokens
// 2 % more.
constexpr int kPagedAhead = 1;
constexpr int kPagedMmaK = 32;     // E4M3 values of a tcgen05.mma
constexpr int kPagedFill = 1024;  // columns of a -inf span
constexpr int32_t kPagedTimeout = 1;           // status bit: a bounded wait gave up
constexpr uint64_t kPagedDrainNs = 1000000000ull;  // bound of the last wait before a CTA gives up
// A suspended thread wakes when its phase completes, or after this (a shorter limit of the wait bounds
// it too) to see whether the wait has run out or another warp has given up.
constexpr uint32_t kPagedSuspendNs = 20000;

// A tile in the ring.
struct alignas(16) PagedItem {
    float scale[kPagedTile];
    int64_t b;
    int32_t tile, row;  // tile -1: the end; row: the CTA's running number of its rows
    int32_t len, pad;
    uint32_t there[4];  // which keys are there; kTma: which pieces, in the first
};

// kTok: tokens of a CTA (1, 2 or 4).
template <int kTok, bool kTma>
struct PagedShape {
    static constexpr int kCopyWarps = kTma ? 1 : 4;
    static constexpr int kMmaWarp = kCopyWarps + kPagedFinishWarps, kFillWarp = kMmaWarp + 1;
    static constexpr int kThreads = 32 * (kFillWarp + 1);
    static constexpr int kStages = kTok == 4 ? 3 : 4;
    // What is known of a tile outlives its keys: when the copies of tile j + kItems begin, tile j + 3 is
    // multiplied, so tile j + 1 is finished, and all finishing warps have seen tile j.
    static constexpr int kItems = kStages + 3;
    static constexpr int kSlots = kTok == 4 ? 3 : 4;  // rows whose Q and w are held
    static constexpr int kCtasPerSm = 2;
    static constexpr uint32_t kN = kTok * kPagedHeads;
    static constexpr uint32_t kTmemCols = 2 * kN;
    static constexpr uint32_t kKBytes = kPagedTile * kPagedDim, kQBytes = kN * kPagedDim;
    static constexpr uint32_t kOffQ = kStages * kKBytes;
    static constexpr uint32_t kOffW = kOffQ + kSlots * kQBytes;
    static constexpr uint32_t kOffItem = kOffW + kSlots * kN * 4;
    static constexpr uint32_t kOffBar = kOffItem + kItems * sizeof(PagedItem);
    // Barriers: stage full, stage empty, item there, buffer full, buffer empty, slot empty.  Nobody may
    // fall a whole phase behind a barrier that it waits for, so the finishing warps wait for the items',
    // not for the stages', which may be filled again before a tile is finished.
    static constexpr int kFull = 0, kEmpty = kStages, kItem = 2 * kStages;
    static constexpr int kAccFull = kItem + kItems, kAccEmpty = kAccFull + 2;
    static constexpr int kSlotEmpty = kAccEmpty + 2, kBars = kSlotEmpty + kSlots;
    static constexpr uint32_t kSmem = kOffBar + 8 * kBars + 1024;  // slack for aligning the base
    // The first tile whose copies onto a ring of `ring` places may be under way when the copy warp stops
    // before tile j, or has ended with it: those of tile i have landed once the copies of tile i + ring
    // begin, and the end takes its places as a tile does.
    __host__ __device__ static constexpr int32_t under_way(int32_t j, bool ended, int32_t ring)
    {
        const int32_t i = j - ring + (ended ? 1 : 0);
        return i > 0 ? i : 0;
    }
    // D f32, A = B = E4M3, both K-major, M = 128 keys
    static constexpr uint32_t kIdesc = (1u << 4) | ((kN >> 3) << 17) | (uint32_t(kPagedTile >> 4) << 24);
};

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

// Two floats' fused multiply-add in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

template <int kTok, bool kTma>
__global__ void __launch_bounds__(PagedShape<kTok, kTma>::kThreads, PagedShape<kTok, kTma>::kCtasPerSm)
    paged_logits_kernel(const __grid_constant__ PagedLogitsParams p,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_q)
{
    using S = PagedShape<kTok, kTma>;
    constexpr int kScanWarps = kPagedScanThreads / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t s_scan[kPagedScanThreads / 32], s_first[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int32_t s_stop;
    uint8_t* const smem =
        smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_addr(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int t0 = blockIdx.y * kTok, n_tok = min(kTok, p.T - t0);
    const int64_t cap = min(p.N, int64_t(p.table.cols) * p.keys.page_size);
    auto bar = [&](int i) { return base + S::kOffBar + 8 * i; };
    PagedItem* const items = reinterpret_cast<PagedItem*>(smem + S::kOffItem);

    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the rows' costs, in units of about half a kilobyte moved
    const int32_t c_tile = 34 + n_tok, c_fill = 8 * n_tok;
    auto full_length = [&](int64_t b) -> int64_t {
        return in_bounds(p.bounds, kMemLens, p.lens + b, 4) ? p.lens[b] : 0;
    };
    auto length = [&](int64_t b) {
        const int64_t n = full_length(b);
        return int32_t(n < 0 ? 0 : n < cap ? n : cap);
    };
    auto tiles = [&](int64_t b) { return (length(b) + kPagedTile - 1) / kPagedTile; };
    auto fills = [&](int32_t n_tiles) {
        const int32_t left = int32_t(p.N) - n_tiles * kPagedTile;
        return !p.clean || left <= 0 ? 0 : (left + kPagedFill - 1) / kPagedFill;
    };
    auto cost = [&](int64_t b) {
        const int32_t n = tiles(b);
        return int64_t(n) * c_tile + int64_t(fills(n)) * c_fill;
    };
    const int64_t per = (p.B + kPagedScanThreads - 1) / kPagedScanThreads;
    int64_t sum = 0, scan = 0;
    if (tid < kPagedScanThreads) {
        const int64_t b1 = min(per * (tid + 1), p.B);
        for (int64_t b = per * tid; b < b1; ++b) sum += cost(b);
        scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t x = __shfl_up_sync(~0u, scan, o);
            if (lane >= o) scan += x;
        }
        if (lane == 31) s_scan[warp] = scan;
    }

    // ---- tensor memory and barriers
    if (warp == S::kMmaWarp) {
        // the permit is given up at once: while a CTA holds it, the SM's next CTA waits in its alloc
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), S::kTmemCols);
        ptx::tmem_relinquish();
        if (lane == 0) {
            for (int i = 0; i < S::kStages; ++i) {
                ptx::mbar_init(bar(S::kFull + i), S::kCopyWarps);
                ptx::mbar_init(bar(S::kEmpty + i), 1);
            }
            for (int i = 0; i < 2; ++i) {
                ptx::mbar_init(bar(S::kAccFull + i), 1);
                ptx::mbar_init(bar(S::kAccEmpty + i), 4);
            }
            for (int i = 0; i < S::kItems; ++i) ptx::mbar_init(bar(S::kItem + i), S::kCopyWarps);
            for (int i = 0; i < S::kSlots; ++i)
                ptx::mbar_init(bar(S::kSlotEmpty + i), kPagedFinishWarps);
            ptx::mbar_init_fence();
            s_stop = 0;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_tmem;
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) {
        if (w == warp) before = total + scan - sum;
        total += s_scan[w];
    }
    const int64_t from = blockIdx.x * total / gridDim.x, to = (blockIdx.x + 1) * total / gridDim.x;
    if (tid < kPagedScanThreads && before <= from && from < before + sum) {
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

    // Waits for a phase of a barrier; false when the CTA gives up.
    auto wait = [&](int i, uint32_t parity) {
        if (ptx::mbar_try_wait(bar(i), parity)) return true;
        const uint64_t start = ptx::globaltimer_ns();
        while (!ptx::mbar_try_wait_sleep(bar(i), parity, p.suspend_ns)) {
            if (s_stop) return false;
            if (ptx::globaltimer_ns() - start > p.wait_ns) {
                s_stop = 1;
                atomicOr(p.status, kPagedTimeout);
                return false;
            }
        }
        return true;
    };
    // Waits for what is under way, whether or not the CTA gives up, for kPagedDrainNs at most.
    auto drain = [&](uint32_t at, uint32_t parity) {
        const uint64_t start = ptx::globaltimer_ns();
        while (!ptx::mbar_try_wait_sleep(at, parity, kPagedSuspendNs) &&
               ptx::globaltimer_ns() - start <= kPagedDrainNs) {
        }
    };
    // The same for all lanes of a warp: they go on or give up together.
    auto wait_warp = [&](int i, uint32_t parity) { return __all_sync(~0u, wait(i, parity)) != 0; };
    // Items i of a share that begin in [from, to), of n items of cost c each from `at` on.
    auto share = [&](int64_t at, int32_t c, int32_t n, int32_t* lo, int32_t* hi) {
        *lo = from > at ? int32_t(min(int64_t(n), (from - at + c - 1) / c)) : 0;
        *hi = to > at ? int32_t(min(int64_t(n), (to - at + c - 1) / c)) : 0;
    };

    if (from >= to) {
        // nothing to do
    } else if (warp < S::kCopyWarps) {
        // ------------------------------------------------------------ copy
        int64_t b = s_first[0], at = s_first[1];  // the next row, the cost before it
        int64_t cur_b = 0;
        int32_t tile = 0, tile_end = 0, len = 0, row = -1;
        bool first = false;
        int32_t page = -1, page_row = 0;
        // Moves on to the next tile and looks up its pages; tile = -1: there is none.
        auto next = [&] {
            ++tile;
            first = false;
            while (tile >= tile_end) {
                if (at >= to) {
                    tile = -1;
                    return;
                }
                cur_b = b++;
                len = length(cur_b);
                const int32_t n = (len + kPagedTile - 1) / kPagedTile;
                share(at, c_tile, n, &tile, &tile_end);
                at += int64_t(n) * c_tile + int64_t(fills(n)) * c_fill;
                first = true;
            }
            if (first) ++row;
            // kTma: a lane's piece, else its key
            const int32_t n = tile * kPagedTile + (kTma ? lane << p.box_shift : tid);
            if (!((!kTma || lane < kPagedTile >> p.box_shift) && n < len &&
                  locate(p.bounds, p.keys, p.table, cur_b, n, &page, &page_row)))
                page = -1;
        };
        int32_t reported = 0;
        auto report = [&](int32_t end) {  // this warp's parts of the tiles before `end` are there
            ptx::fence_proxy_async_smem();
            __syncwarp();
            for (; reported < end; ++reported)
                if (lane == 0) {
                    ptx::mbar_arrive(bar(S::kFull + reported % S::kStages));
                    ptx::mbar_arrive(bar(S::kItem + reported % S::kItems));
                }
        };
        tile = tile_end = 0;
        next();
        int32_t j = 0;
        bool ok = true;
        for (;; ++j) {
            const int stage = j % S::kStages;
            if (j >= S::kStages &&
                !(ok = wait_warp(S::kEmpty + stage, uint32_t(j / S::kStages - 1) & 1u)))
                break;
            PagedItem& item = items[j % S::kItems];
            if (warp == 0 && lane == 0) {
                item.b = cur_b;
                item.tile = tile;
                item.row = row;
                item.len = len;
            }
            if (tile < 0) break;
            if (first) {  // the row's Q and w
                const int slot = row % S::kSlots;
                if (row >= S::kSlots) {
                    const uint32_t parity = uint32_t(row / S::kSlots - 1) & 1u;
                    if (!kTma && !__all_sync(~0u, ptx::mbar_try_wait(bar(S::kSlotEmpty + slot), parity))) {
                        // rows of a tile or two: the slot may wait for tiles not reported yet
                        copy_wait<0>();
                        report(j);
                    }
                    if (!(ok = wait_warp(S::kSlotEmpty + slot, parity))) break;
                }
                const int64_t q0 = (cur_b * p.T + t0) * kPagedHeads;
                for (int i = tid; !kTma && i < n_tok * kPagedHeads * 8; i += 32 * S::kCopyWarps)
                    copy16(base + S::kOffQ + slot * S::kQBytes + i / 8 * 128 + 16 * (i % 8 ^ (i / 8 & 7)),
                           p.q + (q0 + i / 8) * kPagedDim + 16 * (i % 8),
                           in_bounds(p.bounds, kMemQ, p.q + (q0 + i / 8) * kPagedDim + 16 * (i % 8), 16));
                for (int i = tid; !kTma && i < n_tok * kPagedHeads / 4; i += 32 * S::kCopyWarps)
                    copy16(base + S::kOffW + slot * S::kN * 4 + 16 * i, p.w + q0 + 4 * i,
                           in_bounds(p.bounds, kMemW, p.w + q0 + 4 * i, 16));
            }
            if constexpr (kTma) {
                auto piece_row = [&] { return int32_t(uint32_t(page) * p.page_rows + page_row); };
                auto piece_scales = [&] { return p.keys.scale + page * p.keys.scale_page_stride + page_row; };
                const bool have =
                    page >= 0 &&
                    in_bounds(p.bounds, kMemData, p.keys.data + piece_row() * p.keys.row_stride,
                              ((1 << p.box_shift) - 1) * p.keys.row_stride + kPagedDim) &&
                    in_bounds(p.bounds, kMemScale, piece_scales(), 4u << p.box_shift);
                auto first_query = [&] { return (cur_b * p.T + t0) * kPagedHeads; };
                const bool fetch =
                    first &&
                    in_bounds(p.bounds, kMemQ, p.q + first_query() * kPagedDim, n_tok * kPagedHeads * kPagedDim) &&
                    in_bounds(p.bounds, kMemW, p.w + first_query(), n_tok * kPagedHeads * 4);
                const uint32_t pieces = __ballot_sync(~0u, have);
                const int slot = row % S::kSlots;
                const uint32_t full = bar(S::kFull + stage), seen = bar(S::kItem + j % S::kItems);
                const uint32_t n_rows = uint32_t(__popc(pieces)) << p.box_shift;
                if (lane == 0) {
                    item.there[0] = pieces;
                    ptx::mbar_arrive_expect_tx(full, n_rows * kPagedDim + (fetch ? S::kQBytes : 0u));
                    ptx::mbar_arrive_expect_tx(seen, n_rows * 4 + (fetch ? n_tok * kPagedHeads * 4 : 0u));
                }
                __syncwarp();
                if (have) {
                    ptx::tma_load_2d(base + stage * S::kKBytes + (lane << p.box_shift) * kPagedDim, &map_k,
                                     full, 0, piece_row());
                    ptx::bulk_load(ptx::smem_addr(&item.scale[lane << p.box_shift]), piece_scales(),
                                   4u << p.box_shift, seen);
                }
                if (fetch && lane == 31) {
                    const int64_t q0 = first_query();
                    ptx::tma_load_2d(base + S::kOffQ + slot * S::kQBytes, &map_q, full, 0, int32_t(q0));
                    ptx::bulk_load(base + S::kOffW + slot * S::kN * 4, p.w + q0, n_tok * kPagedHeads * 4, seen);
                }
                next();
                continue;
            }
            const float* const at_scale =
                p.keys.scale + (page >= 0 ? int64_t(page) * p.keys.scale_page_stride +
                                                int64_t(page_row) * p.keys.scale_row_stride
                                          : 0);
            const bool there = page >= 0 && in_bounds(p.bounds, kMemScale, at_scale, 4);
            const uint32_t place = there ? page * p.units.page + page_row * p.units.row : kNoRow;
            const uint32_t dst = base + stage * S::kKBytes + warp * 32 * 128;
            const int c = lane % 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + lane / 8;
                const uint32_t src = __shfl_sync(~0u, place, r);
                const uint8_t* const at = p.keys.data + uint64_t(src != kNoRow ? src : 0) * p.units.unit + 16 * c;
                const bool have = src != kNoRow && in_bounds(p.bounds, kMemData, at, 16);
                copy16(dst + r * 128 + 16 * (c ^ (r & 7)), at, have);
            }
            copy4(ptx::smem_addr(&item.scale[tid]), at_scale, there);
            const uint32_t here = __ballot_sync(~0u, there);
            if (lane == 0) item.there[warp] = here;
            copy_commit();
            next();
            copy_wait<kPagedAhead>();
            report(j - kPagedAhead + 1);
        }
        if constexpr (kTma) {
            if (ok && lane == 0) {  // the end
                ptx::mbar_arrive(bar(S::kFull + j % S::kStages));
                ptx::mbar_arrive(bar(S::kItem + j % S::kItems));
            }
            // the copies under way land before this CTA's memory goes, whoever gave up (that a tile has
            // been multiplied says that its keys have landed, not its scales)
            for (int32_t i = S::under_way(j, ok, S::kStages); i < j; ++i)
                drain(bar(S::kFull + i % S::kStages), uint32_t(i / S::kStages) & 1u);
            for (int32_t i = S::under_way(j, ok, S::kItems); i < j; ++i)
                drain(bar(S::kItem + i % S::kItems), uint32_t(i / S::kItems) & 1u);
        } else {
            copy_wait<0>();
            if (ok) report(j + 1);  // the last tiles, and the end
        }
    } else if (warp < S::kMmaWarp) {
        // ------------------------------------------------------------ finish
        // a warp reads the TMEM lanes of its number modulo 4
        const int quarter = warp % 4, parity = (warp - S::kCopyWarps) / 4;
        int32_t row = 0;
        for (int32_t j = 0;; ++j) {
            if (!wait_warp(S::kItem + j % S::kItems, uint32_t(j / S::kItems) & 1u)) break;
            const PagedItem& item = items[j % S::kItems];
            const int32_t tile = item.tile;
            if (tile < 0) break;
            if (item.row != row) {  // the row before is finished with
                if (lane == 0) ptx::mbar_arrive(bar(S::kSlotEmpty + row % S::kSlots));
                row = item.row;
            }
            if ((j & 1) != parity) continue;
            const int64_t b = item.b;
            const int32_t n = tile * kPagedTile + quarter * 32 + lane, len = item.len;
            const float scale = item.scale[quarter * 32 + lane];
            const bool there = kTma ? item.there[0] >> ((quarter * 32 + lane) >> p.box_shift) & 1u
                                    : item.there[quarter] >> lane & 1u;
            const int64_t len_full = full_length(b);
            const float* const w =
                reinterpret_cast<const float*>(smem + S::kOffW) + row % S::kSlots * S::kN;
            float* out = p.out + (b * p.T + t0) * p.ld + n;
            if (!wait_warp(S::kAccFull + (j & 1), uint32_t(j >> 1) & 1u)) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int t = 0; t < kTok; ++t, out += p.ld) {
                if (t >= n_tok) break;
                uint32_t x[kPagedHeads];
                tmem_ld_32(tmem + (uint32_t(quarter * 32) << 16) + (j & 1) * S::kN + t * kPagedHeads, x);
                float2 y0 = make_float2(0.0f, 0.0f), y1 = y0;
#pragma unroll
                for (int h = 0; h < kPagedHeads; h += 4) {
                    const float4 wh = *reinterpret_cast<const float4*>(w + t * kPagedHeads + h);
                    // relu of NaN is NaN, so that it does not pass for data
                    y0 = fma2(make_float2(max_nan(__uint_as_float(x[h]), 0.0f),
                                          max_nan(__uint_as_float(x[h + 1]), 0.0f)),
                              make_float2(wh.x, wh.y), y0);
                    y1 = fma2(make_float2(max_nan(__uint_as_float(x[h + 2]), 0.0f),
                                          max_nan(__uint_as_float(x[h + 3]), 0.0f)),
                              make_float2(wh.z, wh.w), y1);
                }
                const bool seen = n < len && n < len_full - (p.T - 1 - (t0 + t));
                if (n < p.N && (seen || p.clean) && in_bounds(p.bounds, kMemOut, out, 4))
                    __stcs(out, seen && there ? ((y0.x + y0.y) + (y1.x + y1.y)) * scale
                                              : -CUDART_INF_F);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::kAccEmpty + (j & 1)));
        }
    } else if (warp == S::kMmaWarp) {
        // ------------------------------------------------------------ multiply
        if (lane == 0) {
            int32_t j = 0;
            for (;; ++j) {
                const int stage = j % S::kStages;
                if (!wait(S::kFull + stage, uint32_t(j / S::kStages) & 1u)) break;
                const PagedItem& item = items[j % S::kItems];
                if (item.tile < 0) break;
                if (j >= 2 && !wait(S::kAccEmpty + (j & 1), uint32_t((j >> 1) - 1) & 1u)) break;
                ptx::tc_fence_after();
                const uint64_t a = sw128_desc(base + stage * S::kKBytes);
                const uint64_t q = sw128_desc(base + S::kOffQ + item.row % S::kSlots * S::kQBytes);
#pragma unroll
                for (int k = 0; k < kPagedDim / kPagedMmaK; ++k)
                    ptx::mma_f8f6f4(tmem + (j & 1) * S::kN, a + 2ull * k, q + 2ull * k, S::kIdesc,
                                    k > 0 ? 1u : 0u);
                ptx::mma_commit(bar(S::kEmpty + stage));
                ptx::mma_commit(bar(S::kAccFull + (j & 1)));
            }
            // all MMAs are done before their tensor memory is freed
            if (j > 0) drain(bar(S::kAccFull + ((j - 1) & 1)), uint32_t((j - 1) >> 1) & 1u);
        }
        __syncwarp();
    } else if (p.clean) {
        // ------------------------------------------------------------ fill
        int64_t at = s_first[1];
        for (int64_t b = s_first[0]; at < to; ++b) {
            const int32_t n = tiles(b), n_fill = fills(n);
            int32_t lo, hi;
            at += int64_t(n) * c_tile;
            share(at, c_fill, n_fill, &lo, &hi);
            at += int64_t(n_fill) * c_fill;
            if (lo >= hi) continue;
            const int64_t c0 = int64_t(n) * kPagedTile + int64_t(lo) * kPagedFill;
            const int64_t c1 = min(p.N, int64_t(n) * kPagedTile + int64_t(hi) * kPagedFill);
            for (int t = 0; t < n_tok; ++t) {
                float* const out = p.out + (b * p.T + t0 + t) * p.ld;
                // 16-byte stores between the first and the last 16-byte boundary
                const int64_t a0 = min(c1, c0 + int64_t((16u - uint32_t(reinterpret_cast<uintptr_t>(out + c0) & 15u)) % 16u / 4u));
                const int64_t a1 = a0 + (c1 - a0) / 4 * 4;
                if (c0 + lane < a0 && in_bounds(p.bounds, kMemOut, out + c0 + lane, 4))
                    __stcs(out + c0 + lane, -CUDART_INF_F);
#pragma unroll 4
                for (int64_t c = a0 + 4 * lane; c < a1; c += 128)
                    if (in_bounds(p.bounds, kMemOut, out + c, 16))
                        __stcs(reinterpret_cast<float4*>(out + c),
                               make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F));
                if (a1 + lane < c1 && in_bounds(p.bounds, kMemOut, out + a1 + lane, 4))
                    __stcs(out + a1 + lane, -CUDART_INF_F);
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == S::kMmaWarp) ptx::tmem_dealloc(tmem, S::kTmemCols);
}

}  // namespace fp8mqa
