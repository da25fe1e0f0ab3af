// Which channels of a row a block of the gated recurrence takes, and which of them a lane.  A block
// may read the initial state of its channels after another block has written its final state in
// the same place, so no channel may belong to two blocks.
#pragma once
#include <cstdint>

namespace ssm {

struct GChannels {
    int64_t first, end;
};

constexpr int64_t g_groups(int64_t C) { return (C + 63) / 64; }

// 64 channels a group.  Lanes take pairs, and an odd last channel is paired with the one before it;
// where it would be alone in the last group, the group before leaves it that pair.
constexpr GChannels g_channels(int64_t C, int64_t group) {
    const int64_t n = g_groups(C), less = n > 1 && C % 64 == 1 ? 2 : 0;
    return {group * 64 - (group == n - 1 ? less : 0), group == n - 1 ? C : (group + 1) * 64 - (group == n - 2 ? less : 0)};
}

// first channel of pair i (0 .. 31) of the group: past the last pair the last two channels once
// more (of one channel, that one)
constexpr int64_t g_pair(GChannels g, int64_t i) {
    const int64_t c = g.first + 2 * i;
    return c + 1 < g.end ? c : g.end - g.first > 1 ? g.end - 2 : g.first;
}

// channels 0 .. C - 1 each in one group, and no pair across a group's border
constexpr bool g_split_sound(int64_t C) {
    int64_t at = 0;
    for (int64_t group = 0; group < g_groups(C); ++group) {
        const GChannels g = g_channels(C, group);
        if (g.first != at || g.end <= g.first || g.end - g.first > 64) return false;
        for (int64_t i = 0; i < 32; ++i)
            if (g_pair(g, i) < g.first || g_pair(g, i) + (C > 1 ? 1 : 0) >= g.end) return false;
        at = g.end;
    }
    return at == C;
}

}  // namespace ssm
