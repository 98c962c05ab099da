// Where the parts of tree attention's pairs lie.  The rounds of all (sequence, key
// head) pairs form one line, of which every workgroup has a stretch of the same
// length; a pair that crosses borders of stretches leaves a part in each workgroup
// that has some of its rounds.  A workgroup has two places: the pair that its
// stretch begins with uses the first one, a later pair the second.
//
// Plain arithmetic without GPU headers: the join reads what these functions say, and
// a program on the host can check every place that they name.
#pragma once

#include <stdint.h>

namespace sv {

// Rounds of a stretch where `total` (up to 2^31 - 1) are dealt to `groups` workgroups.
constexpr int32_t deal_stretch(int32_t total, int32_t groups) { return total > 0 ? (total - 1) / groups + 1 : 1; }

struct PairParts {
    int32_t group;  // the workgroup that has the first of them
    int32_t count;  // 0: the pair has no rounds
    bool second;    // the first part lies in its workgroup's second place
};

// The parts of a pair whose `rounds` begin at round `from` of the line.
constexpr PairParts pair_parts(int32_t from, int32_t rounds, int32_t stretch)
{
    const int32_t group = from / stretch;
    return PairParts{group, rounds > 0 ? (from + rounds - 1) / stretch - group + 1 : 0, from != group * stretch};
}

// The place of part p < count.
constexpr int64_t part_place(const PairParts& parts, int32_t p)
{
    return (int64_t)(parts.group + p) * 2 + (p == 0 && parts.second ? 1 : 0);
}

// Parts that a lane of the join has on their way at once, where `side` lanes take parts side by side.  None (0) for a pair
// without parts: no place is its own.
constexpr int32_t join_batch(int32_t count, int32_t side)
{
    return count <= 0 ? 0 : count <= 2 * side ? 2 : count <= 4 * side ? 4 : 8;
}

// The part that a lane reads as the p-th (those past the last one read that one and leave it out).
constexpr int32_t join_part(int32_t count, int32_t p) { return p < count ? p : count - 1; }

}  // namespace sv
