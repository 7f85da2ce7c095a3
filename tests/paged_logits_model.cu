// A model of the paged logits' pipeline on the host: its warps take their steps in random order, copies
// land whenever they like, and at some moment warps give up.  Checks what the copy warp waits for before
// the CTA's memory goes: every copy still under way, and no wait that could not end.
#include <cstdio>
#include <random>
#include <vector>

#include "paged_logits_kernel.cuh"

using fp8mqa::PagedShape;

// Phases that a barrier has completed when it holds the given arrivals; a wait for `parity` ends
// if the phase under way has the other one.
static bool wait_ends(int completed, unsigned parity) { return (unsigned(completed) & 1u) != parity; }

template <int kTok>
int run(unsigned seed)
{
    using S = PagedShape<kTok, true>;
    std::mt19937 rng(seed);
    auto pick = [&](int n) { return int(rng() % unsigned(n)); };
    const int n = 1 + pick(4 * S::kItems);
    std::vector<int> row(n);
    const int turn = 1 + pick(4);  // tiles of a row, about
    for (int i = 1; i < n; ++i) row[i] = row[i - 1] + (pick(turn) == 0);
    std::vector<char> keys(n, 0), scales(n, 0), finished(n, 0);
    int j = 0, mma = 0, look[2] = {0, 0}, at_row[2] = {0, 0};
    bool ended = false, stopped = false, frozen_mma = false, frozen[2] = {false, false};
    const int give_up = pick(12 * n + 20);  // the step at which some warps give up
    for (int step = 0; !ended && !stopped; ++step) {
        if (step == give_up) {
            frozen_mma = pick(2);
            frozen[0] = pick(2);
            frozen[1] = pick(2);
        }
        const int what = pick(8);
        if (what < 2) {  // a copy lands, any of those under way
            std::vector<int> open;
            for (int i = 0; i < j; ++i)
                if (!(what ? scales : keys)[i]) open.push_back(i);
            if (!open.empty()) (what ? scales : keys)[open[pick(int(open.size()))]] = 1;
        } else if (what < 4) {  // the copy warp
            const bool first = j < n && (j == 0 || row[j] != row[j - 1]);
            const bool stage = j < S::kStages || mma > j - S::kStages;
            const bool slot = !first || row[j] < S::kSlots ||
                              (at_row[0] > row[j] - S::kSlots && at_row[1] > row[j] - S::kSlots);
            if (!stage || (j < n && !slot)) {
                stopped = step > give_up && pick(4) == 0;  // its wait ran out, or another's did
            } else if (j == n) {
                ended = true;
            } else {
                ++j;
            }
        } else if (what < 6) {  // the multiplying thread
            if (!frozen_mma && mma < j && keys[mma] && (mma < 2 || finished[mma - 2])) ++mma;
        } else {  // the finishing warps of one parity
            const int g = what - 6;
            if (!frozen[g] && look[g] < j && scales[look[g]]) {
                at_row[g] = row[look[g]];
                if (look[g] % 2 == g) {
                    if (mma <= look[g]) continue;
                    finished[look[g]] = 1;
                }
                ++look[g];
            }
        }
    }
    // what is waited for
    std::vector<char> sees_keys(n, 0), sees_scales(n, 0);
    for (int i = S::under_way(j, ended, S::kStages); i < j; ++i) sees_keys[i] = 1;
    for (int i = S::under_way(j, ended, S::kItems); i < j; ++i) sees_scales[i] = 1;
    for (int i = 0; i < j; ++i)
        if ((!keys[i] && !sees_keys[i]) || (!scales[i] && !sees_scales[i])) {
            std::printf("tokens %d seed %u: a copy of tile %d may land after the end at tile %d\n", kTok, seed, i, j);
            return 1;
        }
    // once everything has landed each of these waits ends
    for (int i = 0; i < j; ++i) {
        int full = 0, item = 0;  // phases of tile i's barriers: its place's tiles, and the end
        for (int k = 0; k < j + (ended ? 1 : 0); ++k) {
            full += k % S::kStages == i % S::kStages;
            item += k % S::kItems == i % S::kItems;
        }
        if ((sees_keys[i] && !wait_ends(full, unsigned(i / S::kStages) & 1u)) ||
            (sees_scales[i] && !wait_ends(item, unsigned(i / S::kItems) & 1u))) {
            std::printf("tokens %d seed %u: the wait for tile %d does not end (tile %d)\n", kTok, seed, i, j);
            return 1;
        }
    }
    return 0;
}

int main()
{
    for (unsigned seed = 0; seed < 200000; ++seed)
        if (run<1>(seed) || run<2>(seed) || run<4>(seed)) return 1;
    return 0;
}
