// expert_form.cuh -- what shared memory of a block of expert_few.cuh holds, and how its steps
// go around in it.  (Host code without CUDA's headers: a test compiles it by itself.)
#pragma once

#include <stdint.h>

namespace exl3 {

constexpr int kExpertWarps = 32, kExpertThreads = kExpertWarps * 32, kSets = 4;

// floats from row to row of a block's sums (the step spreads a warp's fragments over all banks)
constexpr int kSumRow = 132;

// TWO: the sets have matrix set % 2 (gate and up) and every second step; otherwise every
// fourth step, whose sums are added under the rows' scales of that step.
// RB: a tile's blocks of 8 rows.  LO: activations are in two parts.
template <int K, int RB, bool LO, bool TWO> struct ExpertForm {
    static constexpr int kMatrices = TWO ? 2 : 1, kGroups = kSets / kMatrices, kRows = RB * 8;
    // inputs of a step: [matrix][64 inputs][part][rows], and the rows' scales
    static constexpr uint32_t kPanel = RB * (LO ? 2u : 1u) * 1024u, kInputs = kMatrices * 2u * kPanel;
    static constexpr uint32_t kZ = kInputs + (TWO ? 0u : 128u);
    // codes of a step of a warp, the ring of `kAhead` of them, and the stages of inputs: what
    // shared memory has room for.  (A warp that is served first takes a step in a third of
    // the latency of memory: two steps in the ring left 36 % of the issue slots empty.)
    static constexpr uint32_t kCodes = 256u * K, kSums = kSets * kRows * kSumRow * 4u;
    static constexpr uint32_t kRoom = 219u * 1024u;
    static constexpr bool fits(int stages, int steps, int meetings) {
        return stages * kZ + steps * kExpertWarps * kCodes + meetings * kSums <= kRoom;
    }
    // (two places for the sums: a tile's rows are read while the next tile's are written)
    static constexpr int kMeet = fits(2 * kGroups, 3, 2) ? 2 : 1;
    static constexpr int kStages = fits(4 * kGroups, 3, kMeet)   ? 4 * kGroups
                                   : fits(3 * kGroups, 3, kMeet) ? 3 * kGroups
                                   : fits(2 * kGroups, 3, kMeet) ? 2 * kGroups
                                                                 : kGroups * 3 / 2;
    static constexpr int kAhead = fits(kStages, 4, kMeet) ? 4 : 3;
    static constexpr uint32_t kRing = kAhead * kCodes;
    static constexpr uint32_t kRingAt = kStages * kZ, kSumsAt = kRingAt + kExpertWarps * kRing;
    static constexpr uint32_t kSmem = kSumsAt + kMeet * kSums + 1024u;

    // Step i of a share is group i % kGroups's.  Its inputs lie in stage i % kStages, and barrier
    // i % kArrivals says that they are there.  A wait tells a barrier's phases apart by one bit, so a
    // warp has to come to every phase of the barriers that it waits on: a barrier's steps are all
    // of one group.  With a stage and a half to a group the groups take turns at a stage, which then
    // has a barrier for each of two.
    static constexpr int kArrivals = kStages % kGroups ? 2 * kStages : kStages;
    static constexpr int stage(int i) { return i % kStages; }
    static constexpr int arrival(int i) { return i % kArrivals; }
    static constexpr uint32_t parity(int i) { return (uint32_t)(i / kArrivals) & 1u; }
    static_assert(kArrivals % kGroups == 0 && kArrivals % kStages == 0, "a barrier for each stage and group");
    static_assert(fits(kStages, kAhead, kMeet) && kSmem <= 220 * 1024 && kRows <= kExpertWarps, "beside 7 KB of other variables, a row a warp");
};

}  // namespace exl3
