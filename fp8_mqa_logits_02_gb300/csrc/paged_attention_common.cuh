// What the paged attention's kernels and their steps share: parameters, shapes, layouts in the rings, fragments.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"
#include "sm103_ptx.cuh"

namespace fp8mqa {

constexpr int kAttnThreads = 128, kAttnWarps = kAttnThreads / 32;
// Steps in a ring, for each warp that shares it, and CTAs of an SM: what fills the shared memory.  Three
// steps and two CTAs take as long on the ragged batch and 5 % longer on selected positions.
constexpr int kAttnStages = 2;
constexpr int kAttnStages4 = 3;  // of E2M1 caches, whose steps are half as large
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
    int32_t same_rows;  // k_units and v_units are alike (E2M1: those of groups and scales too)
    // E2M1: of the groups' and the rows' scales, and whether a step's positions always share a page (with same_rows)
    RowUnits k_group_units, v_group_units, k_scale_units, v_scale_units;
    int32_t whole_steps;
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

// kType: FP8MQA_E4M3, FP8MQA_BF16, FP8MQA_F16 or FP8MQA_E2M1 of the cache.  kNT: eights of heads of a warp.
// kHq: warps that share a ring, for 8 kNT heads each of one key head.
template <int kType, int kDim_, int kNT_, int kHq_>
struct AttnShape {
    static constexpr bool kE4m3 = kType == 0, kBf16 = kType == 1, kE2m1 = kType == 4;
    static constexpr bool kScaled = kE4m3 || kE2m1;    // rows have scales
    static constexpr int kDim = kDim_, kNT = kNT_, kHq = kHq_;
    static constexpr int kHeads = 8 * kNT;             // heads of a warp
    static constexpr int kStages = (kE2m1 ? kAttnStages4 : kAttnStages) * kHq;
    static constexpr int kStep = kScaled ? 32 : 16;    // positions of a warp's step
    static constexpr int kBlocks = kStep / 16;         // of 16 positions
    static constexpr int kRowBytes = kE2m1 ? kDim / 2 : kDim * (kE4m3 ? 1 : 2);
    static constexpr int kGroupBytes = kE2m1 ? kDim / kGroup : 0;  // of a row
    static constexpr int kPieces = kRowBytes / 16;
    static constexpr int kKRows = kStep / 8;           // rows of S^T a lane has
    static constexpr int kVWords = kRowBytes / 32;     // words of a V row a lane has
    static constexpr int kMT = kDim / 16;              // 16-blocks of dim
    // a ring stage: K rows, V rows, their scales, their groups' scales, and which rows are there
    static constexpr int kRows = kStep * kRowBytes;
    static constexpr int kScales = 2 * kRows, kGroups = kScales + (kScaled ? 2 * kStep * 4 : 0);
    static constexpr int kThere = kGroups + 2 * kStep * kGroupBytes;
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
// The same for E2M1 rows of 64 or 32 bytes, of which a lane takes 8 or 4 (a read of V takes them of every
// second of eight rows): rows change places, so that those four rows fill the banks.
template <int kPieces>
__device__ __forceinline__ int v_place4(int r, int c)
{
    return kPieces == 4 ? ((r & ~3) | (r & 1) << 1 | (r >> 1 & 1)) * 4 + (c ^ (r >> 1 & 2))
                        : ((r & ~7) | (r & 1) << 2 | (r >> 1 & 3)) * 2 + c;
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

// What a warp is to do with a row: tiles [lo, hi) of row b, for n_heads query heads (none: <= 0) from h0 on, of key
// head kvh.
struct AttnPart {
    int64_t b;
    int32_t lo, hi;
    int h0, n_heads, kvh, hw, tile;
};

// What comes of it, for the heads 8 nt + 2 t + j: the scores' reference m and the sum l relative to it, and O^T
// relative to the weights' reference w_top (m, but for rows with scales).
template <class S>
struct AttnSums {
    float m[S::kNT][2], l[S::kNT][2], w_top[S::kNT][2], o[S::kNT][S::kMT][4];
};

}  // namespace fp8mqa
