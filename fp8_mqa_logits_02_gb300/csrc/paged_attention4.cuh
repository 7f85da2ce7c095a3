// The steps of attention over an E2M1 cache: a warp's tiles of a row, from its ring into sums.
//
// A row of 128 values is 76 bytes, so at HBM's rate a warp scheduler has 720 instructions for 32 positions
// and 8 query heads, of which the matrix instructions are 32: the rest of a step is what bounds it.
//
//   values      e2m1 * group has 6 significant bits and is exact in f16: one conversion and one product for
//               two values, 256 a step.  K's lanes have 32 (16) values of a row side by side, whole groups;
//               V's have a group's columns of four rows, whose halves of a byte change places so that one
//               conversion gives a column of two rows.
//   copies      where a step's positions share a page (pages of 32, 64, ... rows, every position) the pages of 32
//               steps are looked up at once and a row is some units on from the step's first; the others find each
//               row, as E4M3 steps do.  (Both ways in one loop cost 9 us of 149: the registers of each.)
//   softmax     the weights are computed with the references as they are, which may lag behind the largest
//               score by 2^kAttnLag and more; only where one comes out too large for f16 does the warp look for
//               the largest score, and computes them again.
//
// Rows' scales are as in E4M3 caches: a key's multiplies its scores, a value's its weights, which have a
// reference of their own.
#pragma once

#include <cfloat>

#include "paged_attention_common.cuh"

namespace fp8mqa {

// References before the first score: below every finite one, so that they need no case of their own.
constexpr float kAttnLowest = -FLT_MAX;

// One of two f16 values, twice.
template <int kWhich>
__device__ __forceinline__ uint32_t twice(uint32_t x)
{
    uint32_t r;
    if constexpr (kWhich == 0) asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 %0, {a, a};\n\t}" : "=r"(r) : "r"(x));
    else asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tmov.b32 %0, {b, b};\n\t}" : "=r"(r) : "r"(x));
    return r;
}

// Whether a warp looks up the pages of 32 steps at once where their positions share them.  Not for 16 heads, whose
// registers are short (one row of 131072 positions 23.4 us with it, 22.5 without; a batch with 8 heads a warp 149 and
// 154; a batch with 16 was not measured).
template <class S>
constexpr bool kWholeSteps = S::kNT == 1;

// kWhole: the positions of a step share a page (pages of 32, 64, ... rows, no list of positions), and K's and V's
// strides are alike.
template <bool kWhole, class S>
__device__ __forceinline__ void attn_steps4(const PagedAttentionParams& p, const AttnRows& rows, const AttnPart& part,
                                            uint8_t* ring, AttnSums<S>& sums)
{
    constexpr int kDim = S::kDim, kNT = S::kNT, kHq = S::kHq;
    constexpr int kPer = 32 / S::kPieces;      // rows that one copy instruction brings
    constexpr int kWords = S::kRowBytes / 16;  // words of eight values that a lane has of a K row
    constexpr float kMost = 256.0f;                // 2^kAttnLag
    constexpr uint32_t kMostBits = (15 + 15) << 10;  // 2^(kAttnLag + kAttnLift) in f16
    static_assert(kAttnLag == 8.0f && kAttnLift == 7.0f, "as the two say");
    static_assert(S::kStep == 32, "a lane a position");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int kvh = part.kvh, tile = part.tile, side = part.hw * kHq;
    const int32_t count = rows.count(part.b), len = rows.length(part.b);
    const int32_t step_end = min(count, part.hi * tile);
    const uint32_t ring_at = ptx::smem_addr(ring);

    // ---- Q: word w of this lane has values 2 w and 2 w + 1 of those that it has of a K row
    uint32_t qf[kNT][S::kMT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        const int h = nt * 8 + g;
        const uint16_t* const q = static_cast<const uint16_t*>(p.q) + part.b * p.q_row_stride +
                                  int64_t(part.h0 + h) * p.q_head_stride + t * (kDim / 4);
#pragma unroll
        for (int s = 0; s < S::kMT; s += 2) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (h < part.n_heads && in_bounds(p.bounds, kMemQ, q + 4 * s, 16))
                x = *reinterpret_cast<const uint4*>(q + 4 * s);
            qf[nt][s][0] = x.x;
            qf[nt][s][1] = x.y;
            qf[nt][s + 1][0] = x.z;
            qf[nt][s + 1][1] = x.w;
        }
    }

    // ---- finding a step's rows: lane i has its i-th position.  (A list is read two steps ahead: its load, the table's
    // and the rows' copies hang on one another.)
    const int32_t* const table = p.table.ids + part.b * p.table.stride;
    const int32_t* const listed_at = p.indices + part.b * p.indices_stride;
    int32_t page = -1, row = 0, listed = -1;
    auto list = [&](int32_t i) {
        listed = -1;
        if (p.n_indices >= 0 && i + lane < step_end && in_bounds(p.bounds, kMemIndices, listed_at + i + lane, 4))
            listed = listed_at[i + lane];
    };
    auto find = [&](int32_t i) {  // i: the step's first place in the row's list
        const int32_t n = p.n_indices >= 0 ? listed : i + lane;
        page = -1;
        if (i + lane < step_end && n >= 0 && n < len) {
            const int32_t col = p.table.by_page.of(n);
            row = n - col * p.k.page_size;
            if (in_bounds(p.bounds, kMemTable, table + col, 4)) page = table[col];
        }
        if (p.n_indices >= 0) list(i + tile);
    };

    // ---- copying a step's rows into a stage.  A lane's own part of the addresses: row lane / kPieces and piece
    // lane % kPieces of the data, row `lane` of the scales
    const int piece = lane % S::kPieces, first = warp % kHq * kPer + lane / S::kPieces;
    const uint8_t* const k_lane = p.k.data + kvh * p.k.head_stride + 16 * piece;
    const uint8_t* const v_lane = p.v.data + kvh * p.v.head_stride + 16 * piece;
    const uint8_t* const k_groups = p.k.groups + kvh * p.k.group_head_stride;
    const uint8_t* const v_groups = p.v.groups + kvh * p.v.group_head_stride;
    const float* const k_scales = p.k.scale + kvh * p.k.scale_head_stride;
    const float* const v_scales = p.v.scale + kvh * p.v.scale_head_stride;
    auto far = [&](const RowUnits& u, uint32_t at) { return uint64_t(at) * u.unit; };
    // (of steps that keep to a page, where V's addresses are K's and the way from one to the other)
    const uint8_t* const k_own = k_lane + far(p.k_units, first * p.k_units.row);
    const int64_t v_data_on = v_lane - k_lane, v_groups_on = v_groups - k_groups, v_scales_on = v_scales - k_scales;
    auto data = [&](uint32_t to, int r, const uint8_t* k, const uint8_t* v, bool ok) {
        copy16(to + 16 * k_place<S::kPieces>(r, piece), k, ok && in_bounds(p.bounds, kMemData, k, 16));
        copy16(to + S::kRows + 16 * v_place4<S::kPieces>(r, piece), v, ok && in_bounds(p.bounds, kMemData2, v, 16));
    };
    auto scales = [&](uint32_t to, const uint8_t* kg, const uint8_t* vg, const float* ks, const float* vs, bool ok) {
        auto group = [&](uint32_t at, int kind, const uint8_t* from) {
            if constexpr (S::kGroupBytes == 8) copy8(at, from, ok && in_bounds(p.bounds, kind, from, 8));
            else copy4(at, from, ok && in_bounds(p.bounds, kind, from, 4));
        };
        group(to + S::kGroups + S::kGroupBytes * lane, kMemGroups, kg);
        group(to + S::kGroups + S::kGroupBytes * (S::kStep + lane), kMemGroups2, vg);
        copy4(to + S::kScales + 8 * lane, ks, ok && in_bounds(p.bounds, kMemScale, ks, 4));  // side by side
        copy4(to + S::kScales + 8 * lane + 4, vs, ok && in_bounds(p.bounds, kMemScale2, vs, 4));
    };
    auto copy = [&](int stage) {  // what find() found
        const bool there = uint32_t(page) < uint32_t(p.k.pages);
        const uint32_t here = __ballot_sync(~0u, there);
        const uint32_t to = ring_at + stage * S::kStage;
        const uint32_t pg = there ? page : 0, rw = there ? row : 0;
        auto at = [&](const RowUnits& u) { return pg * u.page + rw * u.row; };
        const uint32_t k_at = at(p.k_units), v_at = at(p.v_units);
        if (!kWholeSteps<S> && p.whole_steps && here == ~0u) {
            const uint64_t step = far(p.k_units, kPer * kHq * p.k_units.row);
            const uint8_t* k = k_own + far(p.k_units, __shfl_sync(~0u, k_at, 0));
#pragma unroll
            for (int j = 0; j < S::kStep / kPer / kHq; ++j, k += step) data(to, first + j * kHq * kPer, k, k + v_data_on, true);
        } else {
#pragma unroll
            for (int j = 0; j < S::kStep / kPer / kHq; ++j) {
                const int r = first + j * kHq * kPer;
                const uint32_t k_row = __shfl_sync(~0u, k_at, r), v_row = __shfl_sync(~0u, v_at, r);
                data(to, r, k_lane + far(p.k_units, k_row), v_lane + far(p.v_units, v_row), here >> r & 1u);
            }
        }
        if (warp % kHq == 0) {
            auto of = [&](auto* from, const RowUnits& u) { return from + far(u, at(u)); };
            scales(to, of(k_groups, p.k_group_units), of(v_groups, p.v_group_units), of(k_scales, p.k_scale_units),
                   of(v_scales, p.v_scale_units), there);
            if (lane == 0) *reinterpret_cast<uint32_t*>(ring + stage * S::kStage + S::kThere) = here;
        }
    };

    // ---- both where steps keep to a page: lane i has the page of the warp's i-th next step, 32 steps ahead, and where
    // the step's first row lies
    const uint8_t* const groups_own = k_groups + far(p.k_group_units, lane * p.k_group_units.row);
    const float* const scales_own = k_scales + far(p.k_scale_units, lane * p.k_scale_units.row);
    uint32_t at_data = 0, at_group = 0, at_scale = 0, valid = 0;
    int turn = 0;
    auto look = [&](uint32_t i) {
        const uint32_t n = i + uint32_t(lane * tile);  // (past 2^31 perhaps)
        page = -1;
        if (n < uint32_t(step_end)) {
            const int32_t* const from = table + p.table.by_page.of(int32_t(n));
            if (in_bounds(p.bounds, kMemTable, from, 4)) page = *from;
        }
    };
    auto find_whole = [&](int32_t i) {
        const bool there = uint32_t(page) < uint32_t(p.k.pages);
        const uint32_t n = min(uint32_t(i) + uint32_t(lane * tile), uint32_t(step_end));
        const uint32_t pg = there ? page : 0, rw = there ? n - p.table.by_page.of(int32_t(n)) * p.k.page_size : 0;
        auto at = [&](const RowUnits& u) { return pg * u.page + rw * u.row; };
        at_data = at(p.k_units);
        at_group = at(p.k_group_units);
        at_scale = at(p.k_scale_units);
        valid = __ballot_sync(~0u, there);
        turn = 0;
        look(uint32_t(i) + uint32_t(32 * tile));
    };
    auto copy_whole = [&](int stage, int32_t i) {
        const uint32_t to = ring_at + stage * S::kStage;
        const uint32_t left = uint32_t(step_end - i);
        const uint32_t here = !(valid >> turn & 1u) ? 0u : left < 32u ? ~(~0u << left) : ~0u;
        uint32_t row_at = __shfl_sync(~0u, at_data, turn);
#pragma unroll
        for (int j = 0; j < S::kStep / kPer / kHq; ++j, row_at += kPer * kHq * p.k_units.row) {
            const int r = first + j * kHq * kPer;
            const uint8_t* const k = k_own + far(p.k_units, row_at);
            data(to, r, k, k + v_data_on, here >> r & 1u);
        }
        if (warp % kHq == 0) {
            const uint8_t* const group = groups_own + far(p.k_group_units, __shfl_sync(~0u, at_group, turn));
            const float* const scale = scales_own + far(p.k_scale_units, __shfl_sync(~0u, at_scale, turn));
            scales(to, group, group + v_groups_on, scale, scale + v_scales_on, here >> lane & 1u);
            if (lane == 0) *reinterpret_cast<uint32_t*>(ring + stage * S::kStage + S::kThere) = here;
        }
    };

    int32_t i0 = part.lo * tile + warp / side * S::kStep;  // the step being computed
    int32_t ahead = i0;                                    // the step that find() found
    if constexpr (kWhole) {
        look(ahead);
        find_whole(ahead);
    } else {
        if (p.n_indices >= 0) list(ahead);
        find(ahead);
    }
    auto fill = [&](int stage) {
        if (ahead < step_end) {
            if constexpr (kWhole) {
                copy_whole(stage, ahead);
                ahead += tile;
                if (++turn == 32) find_whole(ahead);
            } else {
                copy(stage);
                find(ahead += tile);
            }
        }
        copy_commit();
    };
#pragma unroll 1
    for (int j = 0; j < S::kStages - 1; ++j) fill(j);

    // ---- Q as f16 B fragments, each head brought to a largest magnitude of 2^12 .. 2^13 by a power of two (what then
    // falls below f16's range is under 2^-36 of the largest), and each head's factor of the scores, in powers of two
    float factor[kNT][2];
    auto &m = sums.m, &l = sums.l, &w_top = sums.w_top;
    auto& o = sums.o;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        float by = 1.0f;
        if (p.q_bf16) {
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
            const int e = min(max(int(__float_as_uint(top) >> 23), 20), 254) - 139;
            float down = copysignf(__uint_as_float(uint32_t(127 - e) << 23), p.sm_scale);
            if (p.sm_scale != p.sm_scale) down = p.sm_scale;  // NaN in every score of a row that is there
            by = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
            for (int s = 0; s < S::kMT; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    qf[nt][s][j] = pack16<false>(__uint_as_float(qf[nt][s][j] << 16) * down,
                                                 __uint_as_float(qf[nt][s][j] & 0xFFFF0000u) * down);
        }
        else if (!(p.sm_scale >= 0.0f)) {  // (NaN too, as above)
#pragma unroll
            for (int s = 0; s < S::kMT; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) qf[nt][s][j] = p.sm_scale < 0.0f ? qf[nt][s][j] ^ 0x80008000u : 0x7FFF7FFFu;
        }
        // (above 0, so that -inf stays -inf: a scale of 0 counts as one that leaves nothing of the scores)
        const float c = fmaxf(fabsf(p.sm_scale) * 1.4426950408889634f * by, 1e-35f);
        factor[nt][0] = __shfl_sync(~0u, c, 8 * t);
        factor[nt][1] = __shfl_sync(~0u, c, 8 * t + 4);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[nt][j] = w_top[nt][j] = kAttnLowest;
            l[nt][j] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < S::kMT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
    }

#pragma unroll 1
    for (int stage = 0, t_left = part.hi - part.lo; t_left > 0;
         --t_left, i0 += tile, stage = stage + 1 < S::kStages ? stage + 1 : 0) {
        // a ring of one warp: the next copies go out first; a shared one: all its warps' copies
        // are there, and all are done with the stage that the next ones fill
        if (kHq > 1) copy_wait<S::kStages - 2>();
        if (kHq > 1) __syncthreads();  // (two key heads side by side need none: 166 us with it, 155 without)
        fill(stage > 0 ? stage - 1 : S::kStages - 1);
        if (i0 >= step_end || (kHq > 1 && part.n_heads <= 0)) continue;
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
        for (int mb = 0; mb < S::kBlocks; ++mb) {
            uint32_t w[2][kWords], by[2][kWords];  // of rows g and g + 8
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * mb + 8 * i + g;
                const uint8_t* const group = at_k + S::kGroups + r * S::kGroupBytes + t * S::kGroupBytes / 4;
                if constexpr (kWords == 4) {
                    const uint4 y = *reinterpret_cast<const uint4*>(at_k + 16 * k_place<S::kPieces>(r, t));
                    w[i][0] = y.x;
                    w[i][1] = y.y;
                    w[i][2] = y.z;
                    w[i][3] = y.w;
                    const uint32_t two = f16x2_of_e4m3x2(*reinterpret_cast<const uint16_t*>(group));
                    by[i][0] = by[i][1] = twice<0>(two);
                    by[i][2] = by[i][3] = twice<1>(two);
                } else {
                    const uint2 y = *reinterpret_cast<const uint2*>(at_k + r * S::kRowBytes + 8 * t);
                    w[i][0] = y.x;
                    w[i][1] = y.y;
                    by[i][0] = by[i][1] = twice<0>(f16x2_of_e4m3x2(*group));
                }
            }
#pragma unroll
            for (int y = 0; y < kWords; ++y) {
                uint32_t a[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f16_of_e2m1(w[i][y], a[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[i][j] = mul_f16x2(a[i][j], by[i][y]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        mma16816<false>(x[nt][mb], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1],
                                        qf[nt][2 * y + j][0], qf[nt][2 * y + j][1]);
            }
        }

        // ---- softmax: this lane has positions 8 r + g, heads 2 t and 2 t + 1
        float lv[S::kKRows];  // log2 of the rows' value scales
        uint32_t sign[S::kKRows], below = 0;
#pragma unroll
        for (int r = 0; r < S::kKRows; ++r) {
            const float2 by = *reinterpret_cast<const float2*>(at_k + S::kScales + 8 * (8 * r + g));
            lv[r] = log2_fast(fabsf(by.y));
            sign[r] = __float_as_uint(by.y) & 0x80000000u;
            below |= sign[r];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) x[nt][r / 2][r % 2 * 2 + j] *= by.x;
        }
        if (here != ~0u) {
#pragma unroll
            for (int r = 0; r < S::kKRows; ++r)
                if (!(here >> (8 * r + g) & 1u))
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) x[nt][r / 2][r % 2 * 2 + j] = -CUDART_INF_F;
        }
        float sum[kNT][2];          // of 2^(score - m)
        uint32_t pw[kNT][S::kKRows];  // weights, 2^(score + log2 value scale - w_top), of two heads each
        auto weigh = [&] {
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                sum[nt][0] = sum[nt][1] = 0.0f;
                uint32_t most = 0;
#pragma unroll
                for (int r = 0; r < S::kKRows; ++r) {
                    float w[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float y = x[nt][r / 2][r % 2 * 2 + j];
                        sum[nt][j] += exp2_fast(fmaf(y, factor[nt][j], -m[nt][j]));
                        w[j] = exp2_fast(fmaf(y, factor[nt][j], lv[r] - w_top[nt][j]));
                    }
                    pw[nt][r] = pack16<false>(w[0], w[1]);
                    most = __vmaxu2(most, pw[nt][r]);
                }
                // (of four terms of 2^kAttnLag; f16 bits of 2^(kAttnLag + kAttnLift), past which is NaN at last)
                over |= sum[nt][0] > 4.0f * kMost || sum[nt][1] > 4.0f * kMost || (most & 0xFFFFu) > kMostBits ||
                        most >> 16 > kMostBits;
            }
            return over;
        };
        const bool over = weigh();
        if (__any_sync(~0u, over || below != 0)) {
            // the references, from the largest score and from the largest one with the row's value scale in it
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = -CUDART_INF_F, wide = -CUDART_INF_F;
#pragma unroll
                    for (int r = 0; r < S::kKRows; ++r) {
                        const float y = x[nt][r / 2][r % 2 * 2 + j];
                        top = fmaxf(top, y);
                        wide = fmaxf(wide, fmaf(y, factor[nt][j], lv[r]));
                    }
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) {
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                        wide = fmaxf(wide, __shfl_xor_sync(~0u, wide, d));
                    }
                    top = fmaxf(m[nt][j], top * factor[nt][j]);
                    wide = fmaxf(w_top[nt][j], wide - kAttnLift);
                    l[nt][j] *= exp2_fast(m[nt][j] - top);
                    const float c = exp2_fast(w_top[nt][j] - wide);
                    m[nt][j] = top;
                    w_top[nt][j] = wide;
#pragma unroll
                    for (int i = 0; i < S::kMT; ++i) {
                        o[nt][i][j] *= c;
                        o[nt][i][2 + j] *= c;
                    }
                }
            weigh();
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int r = 0; r < S::kKRows; ++r) pw[nt][r] ^= sign[r] | sign[r] >> 16;
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) l[nt][j] += sum[nt][j];

        // ---- O^T += V^T P^T
#pragma unroll
        for (int mb = 0; mb < S::kBlocks; ++mb) {
            uint32_t pf[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                pf[nt][0] = transpose8(pw[nt][2 * mb]);
                pf[nt][1] = transpose8(pw[nt][2 * mb + 1]);
            }
            uint32_t w[4][S::kVWords], group[4];  // of four rows: the lane's columns, and the scale of their group
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = 16 * mb + r / 2 * 8 + 2 * t + r % 2;
                if constexpr (S::kVWords == 2) {
                    const uint2 y =
                        *reinterpret_cast<const uint2*>(at_v + 16 * v_place4<S::kPieces>(key, g / 2) + g % 2 * 8);
                    w[r][0] = y.x;
                    w[r][1] = y.y;
                } else {
                    w[r][0] = *reinterpret_cast<const uint32_t*>(at_v + 16 * v_place4<S::kPieces>(key, g / 4) + g % 4 * 4);
                }
                group[r] = at_k[S::kGroups + (S::kStep + key) * S::kGroupBytes + g * S::kGroupBytes / 8];
            }
            const uint32_t by01 = f16x2_of_e4m3x2(group[0] | group[1] << 8);
            const uint32_t by23 = f16x2_of_e4m3x2(group[2] | group[3] << 8);
#pragma unroll
            for (int y = 0; y < S::kVWords; ++y) {
                // bytes of one column of two rows: columns 0, 2, 4 and 6 of a word's, then 1, 3, 5 and 7
                constexpr uint32_t kLow = 0x0F0F0F0Fu;
                uint32_t a[4][4];
                f16_of_e2m1((w[0][y] & kLow) | (w[1][y] << 4 & ~kLow), a[0]);
                f16_of_e2m1((w[0][y] >> 4 & kLow) | (w[1][y] & ~kLow), a[1]);
                f16_of_e2m1((w[2][y] & kLow) | (w[3][y] << 4 & ~kLow), a[2]);
                f16_of_e2m1((w[2][y] >> 4 & kLow) | (w[3][y] & ~kLow), a[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a0 = mul_f16x2(a[0][j], by01), a1 = mul_f16x2(a[1][j], by01);
                    const uint32_t a2 = mul_f16x2(a[2][j], by23), a3 = mul_f16x2(a[3][j], by23);
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        mma16816<false>(o[nt][4 * y + j], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            }
        }
        if (kHq == 1) __syncwarp();  // the stage may be filled again
    }
}

}  // namespace fp8mqa
