// What the paged-cache kernels share: the device's view of a cache, finding a position's row,
// and conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace fp8mqa {

// Every kernel here may be set up while the kernel before it on the stream still runs, and begins with
// griddepcontrol.wait, after which that kernel's writes are seen.  Its loads are plain ones for that
// reason: read-only loads (__ldg) want data that does not change while the kernel is there at all.

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyMax = 1e-30f;  // the least row maximum that a scale is made from

// E2M1 rows: values 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a sign, two a byte (the first one low), an E4M3 scale for
// each 16 of them (a group) and an fp32 scale for the row: value = data * group * scale.
constexpr int kGroup = 16;
constexpr float kE2m1Top = 2688.0f;  // of data * group: 6 * 448

// A cache as a kernel sees it; data strides in bytes.  `groups` is there for E2M1.
struct PagedView {
    uint8_t* data;
    float* scale;
    uint8_t* groups;
    int64_t page_stride, row_stride, head_stride;
    int64_t scale_page_stride, scale_row_stride, scale_head_stride;
    int64_t group_page_stride, group_row_stride, group_head_stride;
    int32_t pages, page_size, heads;
};

// Division of 0 <= n < 2^31 by a number known before the launch: with 2^bits >= d and
// mul = ceil(2^(31 + bits) / d) (under 2^32), mul * d - 2^(31 + bits) < d <= 2^bits, so
// n * mul >> (31 + bits) is exact.
struct FastDiv {
    uint32_t mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t d)
    {
        uint32_t bits = 0;
        while ((uint64_t(1) << bits) < d) ++bits;
        shift = 31 + bits;
        mul = uint32_t(((uint64_t(1) << shift) + d - 1) / d);
    }
    __device__ __forceinline__ int32_t of(int32_t n) const
    {
        return int32_t(uint64_t(uint32_t(n)) * mul >> shift);
    }
};

struct PageTable {
    const int32_t* ids;
    int64_t stride;
    int32_t cols;
    FastDiv by_page;  // by the cache's page size
};

// A row's place in a cache as a 32-bit number of units of `unit` bytes (a common divisor of the
// page and row strides), so that lanes can hand it to one another in one shuffle.
struct RowUnits {
    uint32_t page, row;  // units a page and a row
    uint32_t unit;       // bytes
};
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

// The bounds-checking build (FP8MQA_DEBUG_BOUNDS) holds every access of a paged kernel to global memory
// against what the call's arguments span, and records the first one outside instead of making it.
enum PagedMemory : int32_t {
    kMemSlots = 1,
    kMemRows,      // rows to be written, keys, then values; as the two below
    kMemRows2,
    kMemData,
    kMemData2,
    kMemScale,
    kMemScale2,
    kMemTable,
    kMemLens,      // or the sequences' starts
    kMemIndices,
    kMemQ,
    kMemW,
    kMemOut,
    kMemOutScale,  // or the log of the softmax's sum
    kMemSplits,
    kMemPartial,
    kMemGroups,    // scales of 16 values
    kMemGroups2,
    kMemPositions,
    kMemFreq,
    kMemWeight,    // a norm's
    kMemWeight2,
    kMemOut2,
    kMemOutScale2,
    kMemFree,      // the stack of free pages
    kMemFreeCount,
    kMemStarts,    // where they are written
    kMemKinds
};
constexpr int32_t kPagedOutside = 2;  // status bit: an access that was not made

struct PagedBounds {
#ifdef FP8MQA_DEBUG_BOUNDS
    int32_t* status;
    uint64_t from[kMemKinds], bytes[kMemKinds];
#endif
};

__device__ __forceinline__ bool in_bounds(const PagedBounds& b, int kind, const void* at, uint64_t n)
{
#ifdef FP8MQA_DEBUG_BOUNDS
    const uint64_t off = reinterpret_cast<uint64_t>(at) - b.from[kind];
    if (off <= b.bytes[kind] && n <= b.bytes[kind] - off) return true;
    atomicOr(b.status, kPagedOutside);
    atomicCAS(reinterpret_cast<unsigned long long*>(b.status + 2), 0ull,
              static_cast<unsigned long long>(kind) << 48 | (off & 0xFFFFFFFFFFFFull));
    return false;
#else
    return true;
#endif
}

// The page and row of position n of sequence b; false if it is not there.
__device__ __forceinline__ bool locate(const PagedBounds& bounds, const PagedView& c, const PageTable& t,
                                       int64_t b, int32_t n, int32_t* page, int32_t* row)
{
    const int32_t col = t.by_page.of(n);
    if (n < 0 || col >= t.cols || !in_bounds(bounds, kMemTable, t.ids + b * t.stride + col, 4)) return false;
    *page = *(t.ids + b * t.stride + col);
    *row = n - col * c.page_size;
    return uint32_t(*page) < uint32_t(c.pages);
}

// Four E4M3 values as f16 values, the first two in *lo: exact.
__device__ __forceinline__ void f16_of_e4m3(uint32_t four, uint32_t* lo, uint32_t* hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(*lo), "=r"(*hi)
        : "r"(four));
}

// Two E4M3 values (the low bytes) as f16 values: exact.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// Eight E2M1 values as f16 values, in order: exact.
__device__ __forceinline__ void f16_of_e2m1(uint32_t eight, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(eight));
}

// Eight values as E2M1, each to the nearest (ties to even), within +-6.
__device__ __forceinline__ uint32_t e2m1_of(const float* x)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <class T>
__device__ __forceinline__ float to_float(T x) { return float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

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

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Asynchronous copies into shared memory; what is not there is filled with zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 8 : 0)
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

}  // namespace fp8mqa
