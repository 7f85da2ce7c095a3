// Attention of one new token per row over a paged cache, all of it or selected positions:
//
//   x_n = sm_scale * q . k_n,   out = sum_n softmax(x)_n v_n,   lse = log sum_n exp(x_n)
//
// Bound: every cached row is read once and used by the few query heads of its group, 4 flops a
// value and head, so the bytes of the cache decide.  What counts is bytes in flight: each warp
// copies its positions' rows asynchronously into a ring of its own in shared memory, kAttnStages
// steps of kStep positions, and reads matrix fragments from it.  (Loads straight into the fragments'
// registers left the kernel waiting for memory: 6.4 of 10 warp-cycles, 3.1 TB/s.)
//
//   S^T [positions x heads] = K Q^T   A = K rows as they lie, B = Q^T.  The contraction runs over
//       dim in any order that K and Q share, so lane (g, t) takes 16-byte pieces of row g.
//   O^T [dim x heads] += V^T P^T      A = V^T, B = P^T.  The rows of O^T may come in any order, so
//       lane (g, t) takes the g-th piece of four rows and interleaves them by byte permutes; P^T is
//       S^T's accumulator transposed 8 x 8 by 8 x 8.
//
// The pieces of a row are permuted in the ring so that both ways of reading are free of bank
// conflicts.
//
// (g = lane / 4, t = lane % 4: the lane's row and column in an m16n8k16 fragment.)  Eight heads
// fill a fragment, so a group's heads are taken 8 or 16 at a time.
//
// E4M3 values become f16 exactly; a row's key scale multiplies its scores, its value scale its
// weights.  Weights are rounded to 16 bits for the second product, which the matrix units want (the fp32
// sum takes them unrounded).  f16 has 11 bits: 2^-11 of a weight at most, an eighth of what rounding
// the result to bfloat16 may cost and as much as rounding it to f16 may.  Its range is used to the top: the
// reference of the weights counts 2^kAttnLift, so that a weight loses bits below 2^-21 of the reference
// only and is 0 below 2^-32.  (With the reference at 1 it was 2^-14 and 2^-25: 32767 positions of weight
// 2^-25.4 next to one of 1 lost a quarter of their part of the result.)  E4M3 weights have the rows' value
// scales in them, 2^(x + log2 scale), and a running maximum of their own, so that this holds whatever the
// scales' size.  Weights over bfloat16 caches are bfloat16, 8 bits (2^-8 of a weight at most), with fp32's
// range.
//
// A CTA's four warps take hw key heads (1 or 2) of the same positions and keep in step: the heads
// of a position lie side by side in memory, and reading them together is what DRAM wants.  Groups of
// more than 16 query heads may be shared out to kHq warps that read one ring, so that the cache's bytes
// reach an SM once for 32 or 64 heads.  The warps left over (4 / (hw kHq)) take further positions.
//
// Measured: 64 rows of up to 20001 positions, 64 query and 8 key heads (1.37 GB) 223 us, 6.2 TB/s of 6.7;
// 16 rows of a 16-bit cache (285 MB) 54 us; 2048 selected of 32768 positions for 64 rows (140 MB in rows
// of 128 bytes anywhere) 43 us; one row of 131072 positions, 32 query heads of one key head, 23.4 us with
// the rows in L2, 24.7 us from HBM, where the steps' latency and the join decide.
//
// Split and join: for each chunk of heads the rows' tiles (the CTA's steps) are laid end to end,
// and its CTAs take equal shares of them; the CTAs of one share number follow one another in the
// grid.  A row that lies in one CTA is finished there; the others' partial (m, l, O) go to the
// workspace, and a second kernel joins them, always in the same order.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"
#include "sm103_ptx.cuh"

namespace fp8mqa {

constexpr int kAttnThreads = 128, kAttnWarps = kAttnThreads / 32;
// Steps in a ring, for each warp that shares it, and CTAs of an SM: what fills the shared memory.  Three
// steps and two CTAs take as long on the ragged batch and 5 % longer on selected positions.
constexpr int kAttnStages = 2;
constexpr int kAttnCtasPerSm = 3;
constexpr int kAttnMaxCtas = 512;  // of one launch
constexpr int64_t kAttnMaxPositions = INT32_MAX - 1024;  // of a row

// Powers of two: how far the weights' reference may lag behind the largest score, and what the reference
// counts for in f16 weights; together they keep to f16's range (2^15 < 65504).
constexpr float kAttnLag = 8.0f;
constexpr float kAttnLift = 7.0f;

// What CTA `me` of a chunk (me > 0) says of the row that its share begins within: the row's parts
// are those of CTAs first .. first + parts - 1.  parts = 0: its share begins with a row.
struct AttnSplit {
    int64_t row;
    int32_t first, parts, first_slot, pad[3];
};

struct PagedAttentionParams {
    const void* q;
    int64_t q_row_stride, q_head_stride;  // elements
    PagedView k, v;
    RowUnits k_units, v_units;
    int32_t same_rows;  // k_units and v_units are alike
    int32_t hw;         // key heads that a CTA's warps take: 1 or 2
    PageTable table;
    const int32_t* lens;
    const int32_t* indices;
    int64_t indices_stride;
    int32_t n_indices;  // -1: every position
    int32_t q_heads;
    int32_t q_bf16;
    int64_t B;
    float sm_scale;
    void* out;
    float* lse;
    float* partial;  // [2 * CTAs][heads of a CTA][dim], then m and l [2 * CTAs][heads of a CTA][2]
    AttnSplit* splits;  // [CTAs of a chunk]
    PagedBounds bounds;
};

// kType: FP8MQA_E4M3, FP8MQA_BF16 or FP8MQA_F16 of the cache.  kNT: eights of heads of a warp.
// kHq: warps that share a ring, for 8 kNT heads each of one key head.
template <int kType, int kDim_, int kNT_, int kHq>
struct AttnShape {
    static constexpr bool kE4m3 = kType == 0, kBf16 = kType == 1;
    static constexpr int kDim = kDim_, kNT = kNT_;
    static constexpr int kHeads = 8 * kNT;             // heads of a warp
    static constexpr int kStages = kAttnStages * kHq;
    static constexpr int kStep = kE4m3 ? 32 : 16;      // positions of a warp's step
    static constexpr int kBlocks = kStep / 16;         // of 16 positions
    static constexpr int kRowBytes = kDim * (kE4m3 ? 1 : 2);
    static constexpr int kPieces = kRowBytes / 16;
    static constexpr int kKRows = kStep / 8;           // rows of S^T a lane has
    static constexpr int kVWords = kRowBytes / 32;     // words of a V row a lane has
    static constexpr int kMT = kDim / 16;              // 16-blocks of dim
    // a ring stage: K rows, V rows, their scales, and which rows are there
    static constexpr int kRows = kStep * kRowBytes;
    static constexpr int kScales = 2 * kRows, kThere = kScales + (kE4m3 ? 2 * kStep * 4 : 0);
    static constexpr int kStage = (kThere + 16 + 127) / 128 * 128;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kAttnWarps / kHq * kRing;
    // a warp's results take the place of its share of the rings
    static constexpr int kResult = kRing / kHq;
    static constexpr int kPitch = kDim + 4;            // floats from head to head: fewer bank conflicts
    static_assert(kHeads * kPitch * 4 <= kResult && kResult % 16 == 0, "room for the results");
};

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float log2_fast(float x)
{
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two floats as 16-bit halves, the first one low.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    uint32_t r;
    if constexpr (kBf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Where piece c of row r lies in a stage.  A fragment read of K takes four pieces of two rows in
// a phase, one of V two pieces of every second of eight rows.
template <int kPieces>
__device__ __forceinline__ int k_place(int r, int c)
{
    return r * kPieces + (kPieces >= 8 ? c ^ ((r & 1) << 2) : c);
}
template <int kPieces>
__device__ __forceinline__ int v_place(int r, int c)
{
    return r * kPieces + (kPieces >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3));
}

// The rows' positions and tiles.
struct AttnRows {
    const PagedAttentionParams& p;
    int64_t cap;
    int32_t tile;  // positions
    __device__ int32_t count(int64_t b) const
    {
        if (p.n_indices >= 0) return p.n_indices;
        return length(b);
    }
    __device__ int32_t length(int64_t b) const
    {
        const int64_t n = in_bounds(p.bounds, kMemLens, p.lens + b, 4) ? p.lens[b] : 0;
        return int32_t(n < 0 ? 0 : n < cap ? n : cap);
    }
    // a row with nothing still has one tile, which writes its empty result
    __device__ int32_t tiles(int64_t b) const { return max(1, (count(b) + tile - 1) / tile); }
};

// Writes float4 number i of a head's result, given the running maximum and sum.
template <int kDim>
__device__ __forceinline__ void attn_store(const PagedAttentionParams& p, int64_t head, int i,
                                           float top, float sum, float4 v)
{
    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
    uint2 two;
    if (p.q_bf16)
        two = make_uint2(pack16<true>(v.x * inv, v.y * inv), pack16<true>(v.z * inv, v.w * inv));
    else
        two = make_uint2(pack16<false>(v.x * inv, v.y * inv), pack16<false>(v.z * inv, v.w * inv));
    uint2* const to = static_cast<uint2*>(p.out) + head * (kDim / 4) + i;
    if (in_bounds(p.bounds, kMemOut, to, 8)) *to = two;
    if (p.lse && i == 0 && in_bounds(p.bounds, kMemOutScale, p.lse + head, 4))
        p.lse[head] = sum == 0.0f ? -CUDART_INF_F : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int kType, int kDim, int kNT, int kHq>
__global__ void __launch_bounds__(kAttnThreads, kAttnCtasPerSm)
    paged_attention_kernel(const __grid_constant__ PagedAttentionParams p)
{
    using S = AttnShape<kType, kDim, kNT, kHq>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_ml[kAttnWarps][S::kHeads][2];
    __shared__ int32_t s_scan[kAttnWarps];
    __shared__ int32_t s_first[2];  // the first row of this CTA, and the tiles before it

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int group = p.q_heads / p.k.heads;
    constexpr int kBlock = kHq * S::kHeads;                  // query heads of a key head in this CTA
    const int parts = (group + kBlock - 1) / kBlock;         // CTAs that a group takes
    const int hw = p.hw, chunks = p.k.heads / hw * parts;
    const int chunk = blockIdx.x % chunks;
    const int me = blockIdx.x / chunks;                      // of the chunk's CTAs
    const int side = hw * kHq;                               // warps at the same positions
    const int kvh = chunk / parts * hw + warp % side / kHq;  // this warp's key head
    const int part0 = chunk % parts * kBlock;                // the CTA's first query head of the group
    const int h_first = part0 + warp % kHq * S::kHeads;      // this warp's
    const int n_heads = min(S::kHeads, group - h_first);     // (none: <= 0)
    const int all_heads = side * S::kHeads;                  // of the CTA, with the empty ones
    const int tile = S::kStep * (kAttnWarps / side);         // positions
    uint8_t* const ring = smem + warp / kHq * S::kRing;
    const uint32_t ring_at = ptx::smem_addr(ring);
    const AttnRows rows{p, int64_t(p.table.cols) * p.k.page_size, tile};

    asm volatile("griddepcontrol.launch_dependents;");  // the join waits for this kernel's end
    asm volatile("griddepcontrol.wait;" ::: "memory");   // and this one for the kernel before it

    // ---- this CTA's share of the tiles (each thread counts those of some consecutive rows)
    const int64_t per = (p.B + kAttnThreads - 1) / kAttnThreads;
    int32_t total, before = 0, mine_sum = 0;  // tiles of all rows, of those before mine, of mine
    if (p.n_indices >= 0) {
        total = int32_t(p.B) * rows.tiles(0);
    } else {
        const int64_t b1 = min(per * (tid + 1), p.B);
        for (int64_t b = per * tid; b < b1; ++b) mine_sum += rows.tiles(b);
        int32_t scan = mine_sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int32_t x = __shfl_up_sync(~0u, scan, o);
            if (lane >= o) scan += x;
        }
        if (lane == 31) s_scan[warp] = scan;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w == warp) before = total + scan - mine_sum;
            total += s_scan[w];
        }
    }
    const int32_t ctas = min(int32_t(gridDim.x) / chunks, total);
    if (me >= ctas) {
        if (chunk == 0 && tid == 0 && in_bounds(p.bounds, kMemSplits, p.splits + me, sizeof(AttnSplit)))
            p.splits[me].parts = 0;
        return;
    }
    // `more` CTAs have each + 1 tiles, the others each
    const int32_t each = total / ctas, more = total - each * ctas;
    auto begin_of = [&](int32_t cta) { return cta * each + min(cta, more); };
    auto owner_of = [&](int32_t t) {
        return t < more * (each + 1) ? t / (each + 1) : more + (t - more * (each + 1)) / each;
    };
    const int32_t first = begin_of(me), end = begin_of(me + 1);
    if (p.n_indices >= 0) {
        if (tid == 0) {
            const int32_t n = rows.tiles(0);
            s_first[0] = first / n;
            s_first[1] = first / n * n;
        }
    } else if (before <= first && first < before + mine_sum) {
        int64_t b = per * tid;
        int32_t at = before;
        for (;; ++b) {
            const int32_t n = rows.tiles(b);
            if (first < at + n) break;
            at += n;
        }
        s_first[0] = int32_t(b);
        s_first[1] = at;
    }
    __syncthreads();
    int64_t b = s_first[0];
    int32_t row_start = s_first[1];

    float* const part_o = p.partial;
    float* const part_ml = p.partial + int64_t(2) * gridDim.x * all_heads * kDim;

    for (int32_t at = first; at < end; ++b) {
        // ---- one segment: tiles [lo, hi) of row b
        const int32_t count = rows.count(b), n_tiles = rows.tiles(b);
        const int32_t lo = at - row_start, hi = min(n_tiles, end - row_start);
        const int h0 = kvh * group + h_first;
        const int32_t len = rows.length(b);

        // ---- Q: the words of this lane's columns, two values each
        uint32_t qf[kNT][S::kMT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int h = nt * 8 + g;
            const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.q_row_stride +
                                int64_t(h0 + h) * p.q_head_stride;
            // word w = 2 s + j (columns of fragment s) is word w % kRun of the run w / kRun of words that
            // lie together, as in the cache's rows: 16 values of 64, or 8 of 32
            constexpr int kRun = S::kE4m3 ? 8 : 4;
#pragma unroll
            for (int w = 0; w < 2 * S::kMT; w += 4) {
                const int d = w / kRun * (8 * kRun) + t * (2 * kRun) + w % kRun * 2;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (h < n_heads && in_bounds(p.bounds, kMemQ, q + d, 16))
                    x = *(reinterpret_cast<const uint4*>(q + d));
                qf[nt][w / 2][0] = x.x;
                qf[nt][w / 2][1] = x.y;
                qf[nt][w / 2 + 1][0] = x.z;
                qf[nt][w / 2 + 1][1] = x.w;
            }
        }

        // ---- a step's rows: lane i finds position i of a step, a step ahead of its copies
        const uint8_t* const k_base = p.k.data + kvh * p.k.head_stride;
        const uint8_t* const v_base = p.v.data + kvh * p.v.head_stride;
        const int32_t step_end = min(count, hi * tile);
        const int mine = lane % S::kStep;
        // (two steps ahead what `indices` says: its load, the table's and the rows' copies hang on
        // one another, and nothing looks at what a load brings before the next one needs it)
        int32_t page = -1, row = 0, listed = -1;
        auto list = [&](int32_t i) {
            listed = -1;
            if (p.n_indices >= 0 && i + mine < step_end) {
                const int32_t* const at = p.indices + b * p.indices_stride + i + mine;
                if (in_bounds(p.bounds, kMemIndices, at, 4)) listed = *at;
            }
        };
        auto find = [&](int32_t i) {  // i: the step's first place in the row's list
            const int32_t n = p.n_indices >= 0 ? listed : i + mine;
            page = -1;
            if (i + mine < step_end && n >= 0 && n < len) {
                const int32_t col = p.table.by_page.of(n);
                row = n - col * p.k.page_size;
                const int32_t* const at = p.table.ids + b * p.table.stride + col;
                if (in_bounds(p.bounds, kMemTable, at, 4)) page = *at;
            }
            list(i + tile);
        };
        auto copy = [&](int stage) {  // the rows that find() found
            const bool there = uint32_t(page) < uint32_t(p.k.pages);
            const uint32_t k_at = there ? page * p.k_units.page + row * p.k_units.row : kNoRow;
            const uint32_t v_at = there ? page * p.v_units.page + row * p.v_units.row : kNoRow;
            const uint32_t to = ring_at + stage * S::kStage;
            constexpr int kPer = 32 / S::kPieces;  // rows in one instruction
            const int c = lane % S::kPieces;
#pragma unroll
            for (int j = 0; j < S::kStep / kPer / kHq; ++j) {
                const int r = (j * kHq + warp % kHq) * kPer + lane / S::kPieces;
                const uint32_t at = __shfl_sync(~0u, k_at, r);
                const uint32_t at2 = p.same_rows ? at : __shfl_sync(~0u, v_at, r);
                const bool ok = at != kNoRow;
                auto k_from = [&] { return k_base + uint64_t(ok ? at : 0) * p.k_units.unit + 16 * c; };
                auto v_from = [&] { return v_base + uint64_t(ok ? at2 : 0) * p.v_units.unit + 16 * c; };
                copy16(to + 16 * k_place<S::kPieces>(r, c), k_from(),
                       ok && in_bounds(p.bounds, kMemData, k_from(), 16));
                copy16(to + S::kRows + 16 * v_place<S::kPieces>(r, c), v_from(),
                       ok && in_bounds(p.bounds, kMemData2, v_from(), 16));
            }
            if (S::kE4m3 && warp % kHq == 0) {
                const int64_t pg = there ? page : 0, rw = there ? row : 0;
                const float* const k_from = p.k.scale + pg * p.k.scale_page_stride +
                                            rw * p.k.scale_row_stride + kvh * p.k.scale_head_stride;
                const float* const v_from = p.v.scale + pg * p.v.scale_page_stride +
                                            rw * p.v.scale_row_stride + kvh * p.v.scale_head_stride;
                copy4(to + S::kScales + 4 * lane, k_from, there && in_bounds(p.bounds, kMemScale, k_from, 4));
                copy4(to + S::kScales + 4 * (S::kStep + lane), v_from,
                      there && in_bounds(p.bounds, kMemScale2, v_from, 4));
            }
            const uint32_t here = __ballot_sync(~0u, there);
            if (lane == 0 && warp % kHq == 0)
                *reinterpret_cast<uint32_t*>(ring + stage * S::kStage + S::kThere) = here;
        };

        int32_t i0 = lo * tile + warp / side * S::kStep;  // the step being computed
        int32_t ahead = i0;                               // the step that find() found
        list(ahead);
        find(ahead);
#pragma unroll 1
        for (int j = 0; j < S::kStages - 1; ++j) {
            if (ahead < step_end) {
                copy(j);
                find(ahead += tile);
            }
            copy_commit();
        }

        // ---- Q as B fragments, and each head's factor of the scores (in powers of two)
        float factor[kNT][2], m[kNT][2], l[kNT][2], w_top[kNT][2], o[kNT][S::kMT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            float by = 1.0f;
            if (S::kE4m3 && p.q_bf16) {
                // bfloat16 -> f16: exact but for the range, so each head is brought to a largest
                // magnitude of 2^12 .. 2^13 by a power of two (what then falls below f16's range
                // is under 2^-36 of the largest)
                float top = 0.0f;
#pragma unroll
                for (int s = 0; s < S::kMT; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        top = fmaxf(top, fabsf(__uint_as_float(qf[nt][s][j] << 16)));
                        top = fmaxf(top, fabsf(__uint_as_float(qf[nt][s][j] & 0xFFFF0000u)));
                    }
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                const int e = min(max(int(__float_as_uint(top) >> 23), 20), 240) - 139;
                const float down = __uint_as_float(uint32_t(127 - e) << 23);
                by = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
                for (int s = 0; s < S::kMT; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        qf[nt][s][j] =
                            pack16<false>(__uint_as_float(qf[nt][s][j] << 16) * down,
                                          __uint_as_float(qf[nt][s][j] & 0xFFFF0000u) * down);
            }
            const float c = p.sm_scale * 1.4426950408889634f * by;
            factor[nt][0] = __shfl_sync(~0u, c, 8 * t);
            factor[nt][1] = __shfl_sync(~0u, c, 8 * t + 4);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = w_top[nt][j] = -CUDART_INF_F;
                l[nt][j] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < S::kMT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
        }

        for (int stage = 0, t_left = hi - lo; t_left > 0;
             --t_left, i0 += tile, stage = (stage + 1) % S::kStages) {
            // a ring of one warp: the next copies go out first; a shared one: all its warps' copies
            // are there, and all are done with the stage that the next ones fill
            if (kHq > 1) copy_wait<S::kStages - 2>();
            if (kHq > 1 || hw > 1) __syncthreads();  // (and the key heads' copies go out together)
            if (ahead < step_end) {
                copy((stage + S::kStages - 1) % S::kStages);
                find(ahead += tile);
            }
            copy_commit();
            if (i0 >= step_end || (kHq > 1 && n_heads <= 0)) continue;
            if (kHq == 1) {
                copy_wait<S::kStages - 1>();
                __syncwarp();
            }
            const uint8_t* const at_k = ring + stage * S::kStage;
            const uint8_t* const at_v = at_k + S::kRows;
            const uint32_t here = *reinterpret_cast<const uint32_t*>(at_k + S::kThere);

            // ---- scores
            float x[kNT][S::kBlocks][4];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int mb = 0; mb < S::kBlocks; ++mb)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[nt][mb][j] = 0.0f;
#pragma unroll
            for (int mb = 0; mb < S::kBlocks; ++mb)
#pragma unroll
                for (int j = 0; j < S::kPieces / 4; ++j) {
                    const int r = 16 * mb + g;
                    const uint4 x0 = *reinterpret_cast<const uint4*>(
                        at_k + 16 * k_place<S::kPieces>(r, 4 * j + t));
                    const uint4 x1 = *reinterpret_cast<const uint4*>(
                        at_k + 16 * k_place<S::kPieces>(r + 8, 4 * j + t));
                    const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w};
                    const uint32_t w1[4] = {x1.x, x1.y, x1.z, x1.w};
                    constexpr int kSteps = S::kE4m3 ? 4 : 2;  // 16 columns of dim each
#pragma unroll
                    for (int y = 0; y < kSteps; ++y) {
                        const int s = j * kSteps + y;
                        uint32_t a0, a1, a2, a3;
                        if constexpr (S::kE4m3) {
                            f16_of_e4m3(w0[y], &a0, &a2);
                            f16_of_e4m3(w1[y], &a1, &a3);
                        } else {
                            a0 = w0[2 * y];
                            a1 = w1[2 * y];
                            a2 = w0[2 * y + 1];
                            a3 = w1[2 * y + 1];
                        }
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma16816<S::kBf16>(x[nt][mb], a0, a1, a2, a3, qf[nt][s][0], qf[nt][s][1]);
                    }
                }

            // ---- softmax: this lane has positions 8r + g, heads 2t and 2t + 1
            float row_lv[S::kKRows];  // log2 of the rows' value scales
            const float* const scales = reinterpret_cast<const float*>(at_k + S::kScales);
            const bool negative = S::kE4m3 && __any_sync(~0u, scales[S::kStep + lane % S::kStep] < 0.0f);
#pragma unroll
            for (int r = 0; r < S::kKRows; ++r) {
                const float row_ks = S::kE4m3 ? scales[r * 8 + g] : 1.0f;
                row_lv[r] = S::kE4m3 ? log2_fast(fabsf(scales[S::kStep + r * 8 + g])) : 0.0f;
                const bool ok = here >> (r * 8 + g) & 1u;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& y = x[nt][r / 2][r % 2 * 2 + j];
                        y = ok ? y * (row_ks * factor[nt][j]) : -CUDART_INF_F;
                    }
            }
            bool moved = false;
            float c[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // the largest score, and (E4M3) the largest score with the row's value scale in it
                    float top = m[nt][j], wide = w_top[nt][j];
#pragma unroll
                    for (int r = 0; r < S::kKRows; ++r) {
                        const float y = x[nt][r / 2][r % 2 * 2 + j];
                        top = fmaxf(top, y);
                        if (S::kE4m3) wide = fmaxf(wide, y + row_lv[r]);
                    }
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) {
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                        if (S::kE4m3) wide = fmaxf(wide, __shfl_xor_sync(~0u, wide, o));
                    }
                    if (!S::kE4m3) wide = top;
                    // what the weights are relative to lags behind the largest score by kAttnLag at most
                    // (weights up to 2^8 are as good), which spares most steps the rescaling of O; not
                    // with bfloat16 weights, where a largest weight of 1 is one that is not rounded
                    // (16 rows of up to 16385: error 2.0e-3, 2.4e-3 with the lag)
                    if constexpr (!S::kBf16) {
                        // (l has the reference of the weights where those are its own terms)
                        if constexpr (!S::kE4m3) top -= kAttnLift;
                        wide -= kAttnLift;
                        if (!(top > m[nt][j] + kAttnLag)) top = m[nt][j];
                        if (!(wide > w_top[nt][j] + kAttnLag)) wide = w_top[nt][j];
                    }
                    const float ref = top == -CUDART_INF_F ? 0.0f : top;
                    const float w_ref = wide == -CUDART_INF_F ? 0.0f : wide;
                    float sum = l[nt][j] * exp2_fast(m[nt][j] - ref);
                    moved |= wide > w_top[nt][j];
                    c[nt][j] = exp2_fast(w_top[nt][j] - w_ref);
                    m[nt][j] = top;
                    w_top[nt][j] = wide;
#pragma unroll
                    for (int r = 0; r < S::kKRows; ++r) {
                        float& y = x[nt][r / 2][r % 2 * 2 + j];
                        const float e = exp2_fast(y - ref);
                        sum += e;
                        y = S::kE4m3 ? exp2_fast(y + row_lv[r] - w_ref) : e;
                        if (S::kE4m3 && negative)
                            y = __uint_as_float(__float_as_uint(y) ^
                                                (__float_as_uint(scales[S::kStep + r * 8 + g]) & 0x80000000u));
                    }
                    l[nt][j] = sum;
                }
            if (__any_sync(~0u, moved)) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int i = 0; i < S::kMT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[nt][i][j] *= c[nt][j % 2];
            }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int mb = 0; mb < S::kBlocks; ++mb) {
                uint32_t pf[kNT][2];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    pf[nt][0] = transpose8(pack16<S::kBf16>(x[nt][mb][0], x[nt][mb][1]));
                    pf[nt][1] = transpose8(pack16<S::kBf16>(x[nt][mb][2], x[nt][mb][3]));
                }
                uint32_t w[4][S::kVWords];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = 16 * mb + r / 2 * 8 + 2 * t + r % 2;
                    if constexpr (S::kVWords == 2) {
                        const uint2 y = *reinterpret_cast<const uint2*>(
                            at_v + 16 * v_place<S::kPieces>(key, g / 2) + g % 2 * 8);
                        w[r][0] = y.x;
                        w[r][1] = y.y;
                    } else {
#pragma unroll
                        for (int j = 0; j < S::kVWords / 4; ++j) {
                            const uint4 y = *reinterpret_cast<const uint4*>(
                                at_v + 16 * v_place<S::kPieces>(key, 8 * j + g));
                            w[r][4 * j] = y.x;
                            w[r][4 * j + 1] = y.y;
                            w[r][4 * j + 2] = y.z;
                            w[r][4 * j + 3] = y.w;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < S::kMT; ++i) {
                    uint32_t a0, a1, a2, a3;
                    if constexpr (S::kE4m3) {
                        const uint32_t sel = i % 2 ? 0x7362 : 0x5140;
                        f16_of_e4m3(__byte_perm(w[0][i / 2], w[1][i / 2], sel), &a0, &a1);
                        f16_of_e4m3(__byte_perm(w[2][i / 2], w[3][i / 2], sel), &a2, &a3);
                    } else {
                        a0 = __byte_perm(w[0][i], w[1][i], 0x5410);
                        a1 = __byte_perm(w[0][i], w[1][i], 0x7632);
                        a2 = __byte_perm(w[2][i], w[3][i], 0x5410);
                        a3 = __byte_perm(w[2][i], w[3][i], 0x7632);
                    }
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        mma16816<S::kBf16>(o[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            }
            if (kHq == 1) __syncwarp();  // the stage may be filled again
        }

        // ---- the warps' results, joined in shared memory
        // [heads][dim], where the rings were
        float* const s_o = reinterpret_cast<float*>(smem + warp * S::kResult);
        if (kHq > 1) __syncthreads();  // nobody reads the rings any more
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // O is counted in 2^w_top, m and l in 2^m
                const float v_back =
                    !S::kE4m3 ? 1.0f : w_top[nt][j] == -CUDART_INF_F ? 0.0f : exp2_fast(w_top[nt][j] - m[nt][j]);
                float sum = l[nt][j];
                sum += __shfl_xor_sync(~0u, sum, 4);
                sum += __shfl_xor_sync(~0u, sum, 8);
                sum += __shfl_xor_sync(~0u, sum, 16);
                const int h = nt * 8 + 2 * t + j;
                if (g == 0) {
                    s_ml[warp][h][0] = m[nt][j];
                    s_ml[warp][h][1] = sum;
                }
                // four columns of a head at a time: those of fragments i and i + 1 lie together
#pragma unroll
                for (int i = 0; i < S::kMT; i += 2) {
                    const int d = S::kE4m3 ? g * (kDim / 8) + 2 * i
                                           : i / 4 * 64 + g * 8 + 2 * i % 8;
                    *reinterpret_cast<float4*>(s_o + h * S::kPitch + d) =
                        make_float4(o[nt][i][j] * v_back, o[nt][i][2 + j] * v_back,
                                    o[nt][i + 1][j] * v_back, o[nt][i + 1][2 + j] * v_back);
                }
            }
        __syncthreads();
        auto finish = [&](int i, int hh, float top, float sum, float4 v) {
            const int h = hh % kBlock;
            if (part0 + h >= group) return;
            attn_store<kDim>(p, b * p.q_heads + (chunk / parts * hw + hh / kBlock) * group + part0 + h,
                             i % (kDim / 4), top, sum, v);
        };
        const bool whole = lo == 0 && hi == n_tiles;
        const int64_t slot = 2 * int64_t(blockIdx.x) + (at == first ? 0 : 1);
        for (int i = tid; i < all_heads * (kDim / 4); i += kAttnThreads) {
            const int hh = i / (kDim / 4), h = hh % S::kHeads;
            float top = -CUDART_INF_F;
            for (int w = hh / S::kHeads; w < kAttnWarps; w += side) top = fmaxf(top, s_ml[w][h][0]);
            const float ref = top == -CUDART_INF_F ? 0.0f : top;
            float sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int w = hh / S::kHeads; w < kAttnWarps; w += side) {
                const float f = exp2_fast(s_ml[w][h][0] - ref);
                const float4 y = *reinterpret_cast<const float4*>(
                    smem + w * S::kResult + (h * S::kPitch + i % (kDim / 4) * 4) * 4);
                sum = fmaf(f, s_ml[w][h][1], sum);
                v.x = fmaf(f, y.x, v.x);
                v.y = fmaf(f, y.y, v.y);
                v.z = fmaf(f, y.z, v.z);
                v.w = fmaf(f, y.w, v.w);
            }
            if (whole) {
                finish(i, hh, top, sum, v);
            } else {
                float4* const to = reinterpret_cast<float4*>(part_o) + slot * (all_heads * (kDim / 4)) + i;
                float2* const to_ml = reinterpret_cast<float2*>(part_ml) + slot * all_heads + hh;
                if (in_bounds(p.bounds, kMemPartial, to, 16)) *to = v;
                if (i % (kDim / 4) == 0 && in_bounds(p.bounds, kMemPartial, to_ml, 8)) *to_ml = make_float2(top, sum);
            }
        }

        // ---- what the second kernel has to know of this row
        if (at == first && chunk == 0 && tid == 0 && me > 0) {
            AttnSplit split;
            split.row = b;
            split.first = owner_of(row_start);
            split.parts = lo == 0 ? 0 : owner_of(row_start + n_tiles - 1) - split.first + 1;
            split.first_slot = begin_of(split.first) == row_start ? 0 : 1;
            if (in_bounds(p.bounds, kMemSplits, p.splits + me, sizeof(split))) p.splits[me] = split;
        }
        at = row_start += hi;
        __syncthreads();  // the results are read: the rings may be filled again
    }
}

// Joins the rows that several CTAs took.  Block (e, k) stands for 8 query heads (k) of share e + 1:
// the row that the share begins within has `parts` shares, so parts - 1 such blocks, which divide the
// 8 heads among them (of 33 shares or more, a quarter of a head's columns each).  A head's partial
// results are divided among the block's warps, and a warp's lanes, so that many loads are under way.
constexpr int kJoinBatch = 8;  // partial results that a lane has under way

// kJoinWarps: 8, or 4, of which six blocks fit on an SM (most of a large grid's blocks find nothing to do).
template <int kDim, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinWarps == 4 ? 6 : 3)
    paged_attention_join_kernel(const __grid_constant__ PagedAttentionParams p, int heads, int ctas)
{
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ __align__(16) float4 s_o[kJoinWarps][kDim / 4];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int group = p.q_heads / p.k.heads, parts = (group + heads - 1) / heads;
    const int chunks = p.k.heads / p.hw * parts, all_heads = p.hw * heads;
    const int chunk = blockIdx.y * 8 / all_heads, first_head = blockIdx.y * 8 % all_heads;
    const int me = blockIdx.x + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!in_bounds(p.bounds, kMemSplits, p.splits + me, sizeof(AttnSplit))) return;
    const AttnSplit split = p.splits[me];
    if (split.parts == 0) return;
    const int n = split.parts, slices = n > 32 ? 4 : 1;
    const int helpers = min(n - 1, 8 * slices), helper = me - split.first - 1;
    if (helper >= helpers) return;
    const int step = helpers / slices;  // this block's heads: helper / slices + j * step
    const int mine = 8 / step + (helper / slices < 8 % step);
    // a power of two of heads at a time, the warps shared out among them
    const int at_once = min(kJoinWarps, mine >= 8 ? 8 : mine >= 4 ? 4 : mine >= 2 ? 2 : 1);
    const int share = kJoinWarps / at_once;
    const int columns = kDim / 4 / slices;                 // float4s of a block's slice: lanes of a member
    const int sub = lane / columns, subs = 32 / columns;   // members at a time
    const int col = helper % slices * columns + lane % columns;
    const float* const part_ml = p.partial + int64_t(2) * ctas * chunks * all_heads * kDim;
    for (int j0 = 0; j0 < mine; j0 += at_once) {
        const int j = j0 + warp / share, r = warp % share;
        const int hh = first_head + helper / slices + j * step;
        float m = -CUDART_INF_F, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < mine) {
            for (int k0 = r * subs + sub; k0 - sub < n; k0 += share * subs * kJoinBatch) {
                float2 ml[kJoinBatch];
                float4 x[kJoinBatch];
#pragma unroll
                for (int i = 0; i < kJoinBatch; ++i) {
                    const int k = k0 + i * share * subs;
                    ml[i] = make_float2(-CUDART_INF_F, 0.0f);
                    x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (k < n) {
                        const int64_t slot = 2 * (int64_t(split.first + k) * chunks + chunk) +
                                             (k == 0 ? split.first_slot : 0);
                        const float2* const from_ml = reinterpret_cast<const float2*>(part_ml) + slot * all_heads + hh;
                        const float4* const from =
                            reinterpret_cast<const float4*>(p.partial + (slot * all_heads + hh) * kDim) + col;
                        if (!in_bounds(p.bounds, kMemPartial, from_ml, 8) || !in_bounds(p.bounds, kMemPartial, from, 16))
                            continue;
                        ml[i] = __ldcg(from_ml);
                        x[i] = __ldcg(from);
                    }
                }
                float top = m;
#pragma unroll
                for (int i = 0; i < kJoinBatch; ++i) top = fmaxf(top, ml[i].x);
                const float ref = top == -CUDART_INF_F ? 0.0f : top, c = exp2_fast(m - ref);
                l *= c;
                o.x *= c;
                o.y *= c;
                o.z *= c;
                o.w *= c;
#pragma unroll
                for (int i = 0; i < kJoinBatch; ++i) {
                    const float f = exp2_fast(ml[i].x - ref);
                    l = fmaf(f, ml[i].y, l);
                    o.x = fmaf(f, x[i].x, o.x);
                    o.y = fmaf(f, x[i].y, o.y);
                    o.z = fmaf(f, x[i].z, o.z);
                    o.w = fmaf(f, x[i].w, o.w);
                }
                m = top;
            }
        }
        for (int s = columns; s < 32; s *= 2) {  // the lanes of the warp's other members
            const float m2 = __shfl_xor_sync(~0u, m, s), top = fmaxf(m, m2);
            const float ref = top == -CUDART_INF_F ? 0.0f : top;
            const float a = exp2_fast(m - ref), b = exp2_fast(m2 - ref);
            // the same sum in the same order in both lanes
            auto both = [&](float x) {
                const float y = __shfl_xor_sync(~0u, x, s);
                return lane & s ? fmaf(b, y, a * x) : fmaf(a, x, b * y);
            };
            l = both(l);
            o = make_float4(both(o.x), both(o.y), both(o.z), both(o.w));
            m = top;
        }
        __syncthreads();
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        if (sub == 0) s_o[warp][lane] = o;
        __syncthreads();
        const int h = hh % heads, part0 = chunk % parts * heads;
        if (j < mine && r == 0 && sub == 0 && part0 + h < group) {
            float top = -CUDART_INF_F;
            for (int w = warp; w < warp + share; ++w) top = fmaxf(top, s_m[w]);
            const float ref = top == -CUDART_INF_F ? 0.0f : top;
            l = 0.0f;
            o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int w = warp; w < warp + share; ++w) {
                const float f = exp2_fast(s_m[w] - ref);
                const float4 x = s_o[w][lane];
                l = fmaf(f, s_l[w], l);
                o.x = fmaf(f, x.x, o.x);
                o.y = fmaf(f, x.y, o.y);
                o.z = fmaf(f, x.z, o.z);
                o.w = fmaf(f, x.w, o.w);
            }
            attn_store<kDim>(p, split.row * p.q_heads + (chunk / parts * p.hw + hh / heads) * group + part0 + h,
                             col, top, l, o);
        }
    }
}

}  // namespace fp8mqa
