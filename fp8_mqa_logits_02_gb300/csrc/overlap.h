// Whether arguments that a call reads and writes share memory.  Host arithmetic on their addresses and strides.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <utility>

namespace fp8mqa {

// n0 blocks, s0 bytes apart, of n1 pieces of `size` bytes, s1 bytes apart.
struct Places {
    const void* at;
    int64_t n0, s0, n1, s1, size;
};

inline Places bytes_at(const void* at, int64_t size) { return {at, 1, 0, 1, 0, at ? size : 0}; }

// Whether two that hold the same things are the same (strides of dimensions of one are never used).
inline bool same_places(const Places& a, const Places& b)
{
    return a.at == b.at && a.n0 == b.n0 && a.n1 == b.n1 && a.size == b.size && (a.n0 <= 1 || a.s0 == b.s0) &&
           (a.n1 <= 1 || a.s1 == b.s1);
}

// Whether no two pieces overlap, as far as one dimension lies within a step of the other.
inline bool apart(const Places& p)
{
    const int64_t s0 = std::abs(p.s0), s1 = std::abs(p.s1);
    auto nest = [&](int64_t n0, int64_t s0, int64_t n1, int64_t s1) {
        return (n1 <= 1 || s1 >= p.size) && (n0 <= 1 || s0 >= (n1 - 1) * s1 + p.size);
    };
    return p.n0 <= 0 || p.n1 <= 0 || p.size <= 0 || nest(p.n0, s0, p.n1, s1) || nest(p.n1, s1, p.n0, s0);
}

// The same bytes with ascending strides, the wider one first, in as few dimensions as they need, within [begin, end).
struct Ascending {
    int64_t begin, end, n0, s0, n1, s1, size;
    Ascending() = default;
    Ascending(const Places& p)
        : begin(reinterpret_cast<intptr_t>(p.at)), n0(p.n0), s0(p.n0 > 1 ? p.s0 : 0), n1(p.n1), s1(p.n1 > 1 ? p.s1 : 0),
          size(p.size)
    {
        if (n0 <= 0 || n1 <= 0 || size <= 0) {
            n0 = n1 = 1;
            s0 = s1 = size = 0;
        }
        if (n0 == 1 && n1 == 1) {
            s0 = s1 = 0;
            end = begin + size;
            return;
        }
        begin += (s0 < 0 ? (n0 - 1) * s0 : 0) + (s1 < 0 ? (n1 - 1) * s1 : 0);
        s0 = std::abs(s0);
        s1 = std::abs(s1);
        if (s0 < s1 || n0 == 1) {
            std::swap(n0, n1);
            std::swap(s0, s1);
        }
        if (n1 > 1 && s1 <= size) {  // no gap between pieces
            size += (n1 - 1) * s1;
            n1 = 1;
            s1 = 0;
        }
        if (n1 > 1 && s0 == n1 * s1) {  // between blocks the same gap as between pieces
            n0 *= n1;
            s0 = s1;
            n1 = 1;
            s1 = 0;
        }
        if (n1 == 1 && n0 > 1 && s0 <= size) {  // no gap between blocks
            size += (n0 - 1) * s0;
            n0 = 1;
            s0 = 0;
        }
        end = begin + (n0 - 1) * s0 + (n1 - 1) * s1 + size;
    }
};

// Whether two share a byte.  Exact where their blocks are as far apart, as those of slices of one tensor are, or few;
// past kOverlapSteps looks, what lies between one another's pieces counts as shared.
constexpr int64_t kOverlapSteps = 1 << 16;
inline bool pieces_meet(Ascending a, Ascending b)
{
    if (a.n0 == 1) a.s0 = b.s0;
    if (b.n0 == 1) b.s0 = a.s0;
    const bool even = a.s0 == b.s0;
    const int64_t blocks = even ? 1 : b.n0;
    if (blocks > kOverlapSteps || a.n1 > kOverlapSteps || b.n1 > kOverlapSteps ||
        a.n1 * b.n1 > kOverlapSteps / blocks)
        return true;
    // a block of a's is `lo` to `hi` steps from its first (or, with even steps, from a block of b's)
    const int64_t lo = even ? 1 - b.n0 : 0, hi = a.n0 - 1;
    for (int64_t k = 0; k < blocks; ++k)
        for (int64_t i = 0; i < a.n1; ++i)
            for (int64_t j = 0; j < b.n1; ++j) {
                // the first step past `from` bytes: does it lie before `to`?
                const int64_t off = b.begin - a.begin + k * b.s0 + j * b.s1 - i * a.s1;
                const int64_t from = off - a.size, to = off + b.size;
                int64_t step = lo;
                if (a.s0 > 0) step = std::max(lo, (from >= 0 ? from / a.s0 : -((-from + a.s0 - 1) / a.s0)) + 1);
                if (step <= hi && step * a.s0 > from && step * a.s0 < to) return true;
            }
    return false;
}
inline bool meet(const Ascending& a, const Ascending& b)
{
    return a.size > 0 && b.size > 0 && a.end > b.begin && b.end > a.begin && pieces_meet(a, b);
}

}  // namespace fp8mqa
