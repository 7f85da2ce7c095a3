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
// weights.  Weights are rounded to 16 bits for the second product (the fp32 sum takes them
// unrounded); their value scales are taken relative to a running power of two, so the largest
// keep their 11 bits whatever the scales' size.
//
// Split and join: the rows' tiles (four warps' steps) are laid end to end, and every CTA takes an
// equal share of them.  A unit (row and head chunk) that lies in one CTA is finished there; the
// others' partial (m, l, O) go to the workspace, and the last CTA of each group of kFan to arrive
// joins the group, then the last group's CTA the groups, always in the same order.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"
#include "sm103_ptx.cuh"

namespace fp8mqa {

constexpr int kAttnThreads = 128, kAttnWarps = kAttnThreads / 32;
constexpr int kAttnStages = 2;     // steps in a warp's ring
constexpr int kAttnCtasPerSm = 3;
constexpr int kAttnMaxCtas = 512;  // of one launch
constexpr int kAttnFan = 16;       // partial results joined at a time
constexpr int kAttnMaxHeads = 16;  // heads a CTA takes at a time
// One launch's arrival counters (zero between launches): a group's and a unit's, by the first
// member's partial slot (two a CTA).
struct AttnCounters {
    int32_t group[2 * kAttnMaxCtas], unit[2 * kAttnMaxCtas];
};

struct PagedAttentionParams {
    const void* q;
    int64_t q_row_stride, q_head_stride;  // elements
    PagedView k, v;
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
    float* partial;  // [2 * CTAs][heads][dim], then m and l [2 * CTAs][heads][2]
    AttnCounters* counters;
};

// kType: FP8MQA_E4M3, FP8MQA_BF16 or FP8MQA_F16 of the cache.
template <int kType, int kDim_, int kNT_>
struct AttnShape {
    static constexpr bool kE4m3 = kType == 0, kBf16 = kType == 1;
    static constexpr int kDim = kDim_, kNT = kNT_;
    static constexpr int kHeads = 8 * kNT;             // heads of a unit
    static constexpr int kStep = kE4m3 ? 32 : 16;      // positions of a warp's step
    static constexpr int kTile = kStep * kAttnWarps;
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
    static constexpr int kRing = kAttnStages * kStage;
    static constexpr int kSmem = kAttnWarps * kRing;
    static_assert(kHeads * kDim * 4 <= kRing, "the warps' results take the rings' place");
};

__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
    return r;
}

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

// Asynchronous copies into shared memory; what is not there is filled with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
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

// Where the rows' tiles lie: row b's tiles, `chunks` units of tiles(b) each, start at
// chunks * (tiles of the rows before it).
template <class S>
struct AttnRows {
    const PagedAttentionParams& p;
    int64_t cap;
    __device__ int32_t count(int64_t b) const
    {
        if (p.n_indices >= 0) return p.n_indices;
        const int64_t n = __ldg(p.lens + b);
        return int32_t(n < 0 ? 0 : n < cap ? n : cap);
    }
    // a row with nothing still has one tile, which writes its empty result
    __device__ int32_t tiles(int64_t b) const { return max(1, (count(b) + S::kTile - 1) / S::kTile); }
};

// Combines n partial results (slots slot(0) .. slot(n - 1)) of a unit's heads; each thread gets
// float4 number i of [heads][dim / 4] with its head's m and l.
template <class S, class Slot, class Use>
__device__ __forceinline__ void attn_join(const float* o, const float* ml, int n, Slot slot, Use use)
{
    for (int i = threadIdx.x; i < S::kHeads * S::kDim / 4; i += kAttnThreads) {
        const int h = i / (S::kDim / 4);
        float top = -CUDART_INF_F;
        for (int k = 0; k < n; ++k) top = fmaxf(top, __ldcg(ml + (slot(k) * S::kHeads + h) * 2));
        float l = 0.0f;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float ref = top == -CUDART_INF_F ? 0.0f : top;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const int64_t at = slot(k);
            const float2 a = __ldcg(reinterpret_cast<const float2*>(ml) + at * S::kHeads + h);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(o) +
                                    at * (S::kHeads * S::kDim / 4) + i);
            const float f = exp2_fast(a.x - ref);
            l = fmaf(f, a.y, l);
            sum.x = fmaf(f, x.x, sum.x);
            sum.y = fmaf(f, x.y, sum.y);
            sum.z = fmaf(f, x.z, sum.z);
            sum.w = fmaf(f, x.w, sum.w);
        }
        use(i, h, top, l, sum);
    }
}

template <int kType, int kDim, int kNT>
__global__ void __launch_bounds__(kAttnThreads, kAttnCtasPerSm)
    paged_attention_kernel(const __grid_constant__ PagedAttentionParams p)
{
    using S = AttnShape<kType, kDim, kNT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_ml[kAttnWarps][S::kHeads][2];
    __shared__ int64_t s_scan[kAttnThreads];
    __shared__ int64_t s_first[2];  // the first row of this CTA, and the tiles before it
    __shared__ int32_t s_last;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int group = p.q_heads / p.k.heads;
    const int parts = (group + S::kHeads - 1) / S::kHeads;  // head chunks of a group
    const int chunks = p.k.heads * parts;
    uint8_t* const ring = smem + warp * S::kRing;
    const uint32_t ring_at = ptx::smem_addr(ring);
    const AttnRows<S> rows{p, int64_t(p.table.cols) * p.k.page_size};

    // ---- this CTA's share of the tiles
    int64_t total;  // tiles of all rows, for one chunk
    if (p.n_indices >= 0) {
        total = p.B * rows.tiles(0);
    } else {
        const int64_t per = (p.B + kAttnThreads - 1) / kAttnThreads;
        const int64_t b0 = min(per * tid, p.B), b1 = min(b0 + per, p.B);
        int64_t sum = 0;
        for (int64_t b = b0; b < b1; ++b) sum += rows.tiles(b);
        s_scan[tid] = sum;
        __syncthreads();
        for (int o = 1; o < kAttnThreads; o *= 2) {
            const int64_t x = tid >= o ? s_scan[tid - o] : 0;
            __syncthreads();
            s_scan[tid] += x;
            __syncthreads();
        }
        total = s_scan[kAttnThreads - 1];
    }
    const int64_t all = total * chunks;
    const int64_t ctas = min(int64_t(gridDim.x), all);
    if (blockIdx.x >= ctas) return;
    const int64_t first = blockIdx.x * all / ctas, end = (blockIdx.x + 1) * all / ctas;
    if (p.n_indices >= 0) {
        if (tid == 0) {
            const int64_t n = rows.tiles(0);
            s_first[0] = first / (n * chunks);
            s_first[1] = s_first[0] * n * chunks;
        }
    } else {
        const int64_t per = (p.B + kAttnThreads - 1) / kAttnThreads;
        int64_t before = (tid ? s_scan[tid - 1] : 0) * chunks;
        if (before <= first && first < s_scan[tid] * chunks) {
            int64_t b = per * tid;
            for (;; ++b) {
                const int64_t n = int64_t(rows.tiles(b)) * chunks;
                if (first < before + n) break;
                before += n;
            }
            s_first[0] = b;
            s_first[1] = before;
        }
    }
    __syncthreads();
    int64_t b = s_first[0], row_start = s_first[1];

    float* const part_o = p.partial;
    float* const part_ml = p.partial + int64_t(2) * gridDim.x * S::kHeads * kDim;

    for (int64_t at = first; at < end;) {
        // ---- one segment: tiles [lo, hi) of unit (b, chunk)
        const int32_t count = rows.count(b), n_tiles = rows.tiles(b);
        if (at >= row_start + int64_t(n_tiles) * chunks) {
            row_start += int64_t(n_tiles) * chunks;
            ++b;
            continue;
        }
        const int chunk = int((at - row_start) / n_tiles);
        const int64_t unit_start = row_start + int64_t(chunk) * n_tiles;
        const int32_t lo = int32_t(at - unit_start);
        const int32_t hi = int32_t(min(int64_t(n_tiles), end - unit_start));
        const int kvh = chunk / parts, h0 = kvh * group + (chunk % parts) * S::kHeads;
        const int n_heads = min(S::kHeads, (kvh + 1) * group - h0);
        const int32_t len = int32_t(min(int64_t(max(__ldg(p.lens + b), 0)), rows.cap));

        // ---- Q as B fragments, and each head's factor of the scores (in powers of two)
        uint32_t qf[kNT][S::kMT][2];
        float factor[kNT][2], m[kNT][2], l[kNT][2], o[kNT][S::kMT][4];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int h = nt * 8 + g;
            const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.q_row_stride +
                                int64_t(h0 + h) * p.q_head_stride;
            // the words of this lane's columns, two values each
            uint32_t raw[S::kMT][2];
#pragma unroll
            for (int s = 0; s < S::kMT; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int d = S::kE4m3 ? s / 4 * 64 + t * 16 + s % 4 * 4 + 2 * j
                                           : (2 * s + j) / 4 * 32 + t * 8 + (2 * s + j) % 4 * 2;
                    raw[s][j] = h < n_heads
                                    ? __ldg(reinterpret_cast<const uint32_t*>(q + d))
                                    : 0u;
                }
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
                        top = fmaxf(top, fabsf(__uint_as_float(raw[s][j] << 16)));
                        top = fmaxf(top, fabsf(__uint_as_float(raw[s][j] & 0xFFFF0000u)));
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
                        raw[s][j] = pack16<false>(__uint_as_float(raw[s][j] << 16) * down,
                                                  __uint_as_float(raw[s][j] & 0xFFFF0000u) * down);
            }
#pragma unroll
            for (int s = 0; s < S::kMT; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) qf[nt][s][j] = raw[s][j];
            const float c = p.sm_scale * 1.4426950408889634f * by;
            factor[nt][0] = __shfl_sync(~0u, c, 8 * t);
            factor[nt][1] = __shfl_sync(~0u, c, 8 * t + 4);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = -CUDART_INF_F;
                l[nt][j] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < S::kMT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
        }
        int32_t v_exp = 1;  // value scales are taken relative to 2^(v_exp - 127)

        // ---- a step's rows: lane i finds position i of a step, a step ahead of its copies
        const uint8_t* const k_base = p.k.data + kvh * p.k.head_stride;
        const uint8_t* const v_base = p.v.data + kvh * p.v.head_stride;
        const int32_t step_end = min(count, hi * S::kTile);
        const int mine = lane % S::kStep;
        int32_t page = -1, row = 0;
        auto find = [&](int32_t i) {  // i: the step's first place in the row's list
            page = -1;
            i += mine;
            if (i < step_end) {
                int32_t n = i;
                if (p.n_indices >= 0) n = __ldg(p.indices + b * p.indices_stride + i);
                if (!(n >= 0 && n < len && locate(p.k, p.table, b, n, &page, &row))) page = -1;
            }
        };
        auto copy = [&](int stage) {  // the rows that find() found
            const bool there = page >= 0;
            const int64_t k_at = there ? page * p.k.page_stride + row * p.k.row_stride : -1;
            const int64_t v_at = there ? page * p.v.page_stride + row * p.v.row_stride : -1;
            const uint32_t to = ring_at + stage * S::kStage;
            constexpr int kPer = 32 / S::kPieces;  // rows in one instruction
            const int c = lane % S::kPieces;
#pragma unroll
            for (int j = 0; j < S::kStep / kPer; ++j) {
                const int r = j * kPer + lane / S::kPieces;
                const int64_t off = __shfl_sync(~0u, k_at, r);
                copy16(to + 16 * k_place<S::kPieces>(r, c), k_base + (off < 0 ? 0 : off) + 16 * c,
                       off >= 0);
            }
#pragma unroll
            for (int j = 0; j < S::kStep / kPer; ++j) {
                const int r = j * kPer + lane / S::kPieces;
                const int64_t off = __shfl_sync(~0u, v_at, r);
                copy16(to + S::kRows + 16 * v_place<S::kPieces>(r, c),
                       v_base + (off < 0 ? 0 : off) + 16 * c, off >= 0);
            }
            if constexpr (S::kE4m3) {
                const int64_t pg = there ? page : 0, rw = there ? row : 0;
                copy4(to + S::kScales + 4 * lane,
                      p.k.scale + pg * p.k.scale_page_stride + rw * p.k.scale_row_stride +
                          kvh * p.k.scale_head_stride,
                      there);
                copy4(to + S::kScales + 4 * (S::kStep + lane),
                      p.v.scale + pg * p.v.scale_page_stride + rw * p.v.scale_row_stride +
                          kvh * p.v.scale_head_stride,
                      there);
            }
            const uint32_t here = __ballot_sync(~0u, there);
            if (lane == 0) *reinterpret_cast<uint32_t*>(ring + stage * S::kStage + S::kThere) = here;
        };

        int32_t i0 = lo * S::kTile + warp * S::kStep;  // the step being computed
        int32_t ahead = i0;                            // the step that find() found
        find(ahead);
#pragma unroll
        for (int j = 0; j < kAttnStages - 1; ++j) {
            if (ahead < step_end) {
                copy(j);
                find(ahead += S::kTile);
            }
            copy_commit();
        }
        for (int stage = 0; i0 < step_end; i0 += S::kTile, stage = (stage + 1) % kAttnStages) {
            if (ahead < step_end) {
                copy((stage + kAttnStages - 1) % kAttnStages);
                find(ahead += S::kTile);
            }
            copy_commit();
            copy_wait<kAttnStages - 1>();
            __syncwarp();
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
                            a0 = f16_of_e4m3(w0[y]);
                            a1 = f16_of_e4m3(w1[y]);
                            a2 = f16_of_e4m3(w0[y] >> 16);
                            a3 = f16_of_e4m3(w1[y] >> 16);
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
            float row_vs[S::kKRows];
            const float* const scales = reinterpret_cast<const float*>(at_k + S::kScales);
#pragma unroll
            for (int r = 0; r < S::kKRows; ++r) {
                const float row_ks = S::kE4m3 ? scales[r * 8 + g] : 1.0f;
                row_vs[r] = S::kE4m3 ? scales[S::kStep + r * 8 + g] : 1.0f;
                const bool ok = here >> (r * 8 + g) & 1u;
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& y = x[nt][r / 2][r % 2 * 2 + j];
                        y = ok ? y * (row_ks * factor[nt][j]) : -CUDART_INF_F;
                    }
            }
            float c_v = 1.0f, v_inv = 1.0f;
            bool moved = false;
            if constexpr (S::kE4m3) {
                const uint32_t top =
                    __reduce_max_sync(~0u, __float_as_uint(scales[S::kStep + lane]) & 0x7FFFFFFFu);
                const int32_t e = min(max(int32_t(top >> 23), v_exp), 253);
                if (e > v_exp) {
                    c_v = exp2_fast(float(v_exp - e));
                    v_exp = e;
                    moved = true;
                }
                v_inv = __uint_as_float(uint32_t(254 - v_exp) << 23);
            }
            float c[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = m[nt][j];
#pragma unroll
                    for (int r = 0; r < S::kKRows; ++r) top = fmaxf(top, x[nt][r / 2][r % 2 * 2 + j]);
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                    moved |= top > m[nt][j];
                    const float ref = top == -CUDART_INF_F ? 0.0f : top;
                    c[nt][j] = exp2_fast(m[nt][j] - ref);
                    m[nt][j] = top;
                    float sum = l[nt][j] * c[nt][j];
#pragma unroll
                    for (int r = 0; r < S::kKRows; ++r) {
                        float& y = x[nt][r / 2][r % 2 * 2 + j];
                        y = exp2_fast(y - ref);
                        sum += y;
                        if (S::kE4m3) y *= row_vs[r] * v_inv;
                    }
                    l[nt][j] = sum;
                }
            if (__any_sync(~0u, moved)) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int i = 0; i < S::kMT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[nt][i][j] *= c[nt][j % 2] * c_v;
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
                        const uint32_t lo2 = __byte_perm(w[0][i / 2], w[1][i / 2], sel);
                        const uint32_t hi2 = __byte_perm(w[2][i / 2], w[3][i / 2], sel);
                        a0 = f16_of_e4m3(lo2);
                        a1 = f16_of_e4m3(lo2 >> 16);
                        a2 = f16_of_e4m3(hi2);
                        a3 = f16_of_e4m3(hi2 >> 16);
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
            __syncwarp();  // the stage may be filled again
        }

        // ---- the warps' results, joined in shared memory
        const float v_back = S::kE4m3 ? __uint_as_float(uint32_t(v_exp) << 23) : 1.0f;
        float* const s_o = reinterpret_cast<float*>(ring);  // [heads][dim], where the ring was
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sum = l[nt][j];
                sum += __shfl_xor_sync(~0u, sum, 4);
                sum += __shfl_xor_sync(~0u, sum, 8);
                sum += __shfl_xor_sync(~0u, sum, 16);
                const int h = nt * 8 + 2 * t + j;
                if (g == 0) {
                    s_ml[warp][h][0] = m[nt][j];
                    s_ml[warp][h][1] = sum;
                }
#pragma unroll
                for (int i = 0; i < S::kMT; ++i) {
                    const int d = S::kE4m3 ? g * (kDim / 8) + 2 * i
                                           : i / 4 * 64 + g * 8 + 2 * i % 8;
                    s_o[h * kDim + d] = o[nt][i][j] * v_back;
                    s_o[h * kDim + d + 1] = o[nt][i][2 + j] * v_back;
                }
            }
        __syncthreads();
        auto finish = [&](int i, int h, float top, float sum, float4 v) {
            if (h >= n_heads) return;
            const int64_t head = b * p.q_heads + h0 + h;
            const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
            const int64_t at4 = head * (kDim / 4) + i % (kDim / 4);
            uint2 two;
            if (p.q_bf16)
                two = make_uint2(pack16<true>(v.x * inv, v.y * inv), pack16<true>(v.z * inv, v.w * inv));
            else
                two = make_uint2(pack16<false>(v.x * inv, v.y * inv), pack16<false>(v.z * inv, v.w * inv));
            static_cast<uint2*>(p.out)[at4] = two;
            if (p.lse && i % (kDim / 4) == 0)
                p.lse[head] = sum == 0.0f ? -CUDART_INF_F
                                          : (top + log2f(sum)) * 0.6931471805599453f;
        };
        const bool whole = lo == 0 && hi == n_tiles;
        const int64_t slot = 2 * int64_t(blockIdx.x) + (at == first ? 0 : 1);
        for (int i = tid; i < S::kHeads * kDim / 4; i += kAttnThreads) {
            const int h = i / (kDim / 4);
            float top = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_ml[w][h][0]);
            const float ref = top == -CUDART_INF_F ? 0.0f : top;
            float sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = exp2_fast(s_ml[w][h][0] - ref);
                const float4 y = reinterpret_cast<const float4*>(smem + w * S::kRing)[i];
                sum = fmaf(f, s_ml[w][h][1], sum);
                v.x = fmaf(f, y.x, v.x);
                v.y = fmaf(f, y.y, v.y);
                v.z = fmaf(f, y.z, v.z);
                v.w = fmaf(f, y.w, v.w);
            }
            if (whole) {
                finish(i, h, top, sum, v);
            } else {
                reinterpret_cast<float4*>(part_o)[slot * (S::kHeads * kDim / 4) + i] = v;
                if (i % (kDim / 4) == 0)
                    reinterpret_cast<float2*>(part_ml)[slot * S::kHeads + h] = make_float2(top, sum);
            }
        }

        // ---- the CTAs' results, joined by whoever arrives last
        if (!whole) {
            // the unit's CTAs are p0 .. p1; the first one's part is its last segment
            const int64_t p0 = ((unit_start + 1) * ctas - 1) / all;
            const int64_t p1 = ((unit_start + n_tiles) * ctas - 1) / all;
            const int n = int(p1 - p0) + 1, me = int(blockIdx.x - p0);
            const int64_t slot0 = 2 * p0 + (p0 * all / ctas == unit_start ? 0 : 1);
            auto slot_of = [&](int k) { return k == 0 ? slot0 : 2 * (p0 + k); };
            auto arrive = [&](int32_t* counter, int expected) {  // true in the last CTA to arrive
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    const bool last = atomicAdd(counter, 1) == expected - 1;
                    if (last) *counter = 0;
                    s_last = last;
                }
                __syncthreads();
                const bool last = s_last;
                if (last) __threadfence();
                return last;
            };
            const int groups = (n + kAttnFan - 1) / kAttnFan;
            const int k0 = me / kAttnFan * kAttnFan, members = min(kAttnFan, n - k0);
            if (arrive(&p.counters->group[slot_of(k0)], members)) {
                if (groups == 1) {
                    attn_join<S>(part_o, part_ml, n, slot_of, finish);
                } else {
                    // the group's sum takes its first member's place
                    const int64_t to = slot_of(k0);
                    float2 ml[S::kHeads * kDim / 4 / kAttnThreads];
                    int c = 0;
                    attn_join<S>(part_o, part_ml, members, [&](int k) { return slot_of(k0 + k); },
                                 [&](int i, int, float top, float sum, float4 v) {
                                     reinterpret_cast<float4*>(part_o)[to * (S::kHeads * kDim / 4) + i] = v;
                                     ml[c++] = make_float2(top, sum);
                                 });
                    __syncthreads();  // every thread has read the first member's m and l
                    c = 0;
                    for (int i = tid; i < S::kHeads * kDim / 4; i += kAttnThreads, ++c)
                        if (i % (kDim / 4) == 0)
                            reinterpret_cast<float2*>(part_ml)[to * S::kHeads + i / (kDim / 4)] = ml[c];
                    if (arrive(&p.counters->unit[slot0], groups))
                        attn_join<S>(part_o, part_ml, groups,
                                     [&](int k) { return slot_of(k * kAttnFan); }, finish);
                }
            }
        }
        at = unit_start + hi;
        __syncthreads();  // the results are read: the rings may be filled again
    }
}

}  // namespace fp8mqa
