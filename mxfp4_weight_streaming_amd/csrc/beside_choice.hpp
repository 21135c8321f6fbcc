// beside_choice.hpp -- how the log probabilities and the adapters split their
// work, by sizes alone.  Plain C++: a host program asks the same rules.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "around_choice.hpp"
#include "around_types.hpp"

namespace moe {

// ---- log probabilities -----------------------------------------------------------
// A workgroup walks a row in segments of kLogprobSegment logits.  Few rows are
// split into parts, a workgroup each, joined by a second kernel.
constexpr int kLogprobMaxParts = 64;            // one lane each where they are joined
constexpr int kLogprobMaxGroups = 40;           // of 256 threads: 40 KB of LDS
constexpr int64_t kLogprobSplitRows = 512;      // fewer rows than this are split

struct LogprobPlan {
    int segments, group_segments, groups, parts, part_segments;
};

constexpr LogprobPlan logprob_plan(int64_t M, int V)
{
    LogprobPlan p{};
    p.segments = (int)ceil_div(V, kLogprobSegment);
    p.group_segments = (int)ceil_div(p.segments, kLogprobMaxGroups);
    p.groups = (int)ceil_div(p.segments, p.group_segments);
    int64_t parts = M <= kLogprobSplitRows ? std::min<int64_t>(ceil_div(2048, M), kLogprobMaxParts) : 1;
    parts = std::min<int64_t>(parts, p.groups);
    p.part_segments = (int)ceil_div(p.groups, parts) * p.group_segments;   // whole groups
    p.parts = (int)ceil_div(p.segments, p.part_segments);
    return p;
}

}  // namespace moe
