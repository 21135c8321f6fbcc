// beside_choice.hpp -- how the log probabilities and the adapters split their
// work, by sizes alone.  Plain C++: a host program asks the same rules.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "around_choice.hpp"
#include "around_types.hpp"

namespace moe {

// ---- log probabilities -----------------------------------------------------------
// Each wave walks a row 1,024 logits at a time.  Short rows have a wave or, with
// alternatives, two each.  Against a workgroup a row, fp32, 5 alternatives, us:
//   logits          2,048        4,096        6,000        8,192
//   16 rows        6.0 /  8.4   8.6 /  8.5  11.2 /  9.3  12.4 /  8.9
//   512            6.3 /  9.7   9.0 / 10.0  12.5 / 11.6  13.4 / 11.3
//   1,024          6.9 / 11.8   9.9 / 12.1  14.5 / 16.3  15.2 / 18.1
//   4,096         16.5 / 38.4  26.4 / 41.3  39.4 / 51.5  55.0 / 51.2
constexpr bool logprob_short(int64_t M, int V) { return V <= 2048 || (V <= 4096 && M >= 512) || (V <= 6144 && M >= 1024); }

// Other rows have a workgroup of 256, 512 or 1,024 threads each, the most with
// which all rows' waves are resident at once, 16 a compute unit (32,768 logits,
// 256 / 512 / 1,024 threads: 256 rows 19.8 / 15.6 / 16.9 us, 512 22.9 / 22.1 /
// 30.7, 1,024 31.7 / 37.8 / 55.6).
constexpr int64_t kLogprobWaves = 16 * kCus;

// Few long rows are split into parts of 256 threads, joined by a second kernel:
// split / a workgroup a row, us:
//   rows             4            64           128          256
//   8,192 logits    9.3 /  8.4   9.9 /  8.8  10.2 /  8.8  10.8 /  9.0
//   20,000          9.4 / 10.2  10.6 / 11.1  11.4 / 11.3  13.9 / 12.1
//   157,184         9.9 / 25.3  19.4 / 28.8  26.3 / 29.7  38.4 / 35.3
constexpr int64_t kLogprobSplitRows = 128;
constexpr int kLogprobSplitLogits = 16 * 1024;
constexpr int64_t kLogprobSplit = 1024;         // workgroups in all
constexpr int kLogprobMaxParts = 64;            // one lane each where they are joined
// Threads that join a row (one of 157,184, 20 alternatives: 256 11.5 us, 512
// 10.4, 1,024 10.1).
constexpr int kLogprobJoin = 1024;

struct LogprobPlan {
    int threads, segments, group_segments, groups, parts, part_segments;   // threads 64: the short rows' kernel
};

constexpr LogprobPlan logprob_plan(int64_t M, int V)
{
    LogprobPlan p{};
    p.threads = 64;
    p.parts = 1;
    p.segments = (int)ceil_div(V, 1024);
    if (logprob_short(M, V)) return p;
    const bool split = M <= kLogprobSplitRows && V > kLogprobSplitLogits;
    p.threads = 256;
    // (no more waves than there are segments for)
    while (!split && p.threads < 1024 && M * p.threads / 64 * 2 <= kLogprobWaves && V > 16 * p.threads) p.threads *= 2;
    p.segments = (int)ceil_div(V, 16 * p.threads);
    // the groups' maxima end up in registers: 64 times 256 of a row in parts, 16 a
    // thread of one that has just been walked
    p.group_segments = (int)ceil_div(p.segments, split ? kLogprobMaxParts : 16);
    p.groups = (int)ceil_div(p.segments, p.group_segments);
    const int64_t parts = split ? std::min<int64_t>({ceil_div(kLogprobSplit, M), kLogprobMaxParts, p.groups}) : 1;
    p.part_segments = (int)ceil_div(p.groups, parts) * p.group_segments;   // whole groups
    p.parts = (int)ceil_div(p.segments, p.part_segments);
    return p;
}

// ---- adapters ------------------------------------------------------------------
constexpr int lora_padded(int r) { return (r + 31) / 32 * 32; }   // ranks of a row of u

// Few tokens: each reads its adapter by itself, where the tokens' ranks are few
// and what all of them read from the caches is at most some 100 MB.  On the
// matrix cores tokens of one adapter share its rows, but a tile of 16 tokens takes
// its adapters in turn.  K = N = 2,560, rank 16, us of few tokens / matrix cores:
//   tokens        64          128         256         512         1,024
//   an adapter    5.7 /  8.0  6.1 /  8.0  7.4 /  8.1 10.2 /  8.5  15.9 /  9.6
//   one for 16    5.8 /  8.0  6.1 /  8.0  7.3 /  8.2 12.9 /  8.6  21.6 /  9.6
//   one each      5.6 / 11.5  6.1 / 14.6 11.5 / 18.4 17.6 / 25.8  29.8 / 39.6
// (1,024 tokens of 8 adapters in any order: 19 on the matrix cores.)  By what they
// read, an adapter / one for 16 / one each:
//   60 tokens, rank 128, 3,300 to 3,400 (103 MB)  11.8 / 12.3  11.7 / 12.6  21.6 / 30.4
//   120, rank 128, 2,560 to 2,560 (157 MB)        11.9 / 10.0  15.4 / 10.2  27.2 / 36.2
//   250, rank 64, 4,096 to 4,096 (262 MB)         18.9 / 11.2  22.1 / 12.0  43.7 / 45.7
constexpr int64_t kLoraFewValues = 16384;      // tokens times their padded rank
constexpr int64_t kLoraFewReads = 48 << 20;    // values of A and B

// Few tokens' workgroups of the same channels on one XCD, so that tokens of one
// adapter find B in its cache: 8 tokens of one adapter, rank 16, 157,184 channels
// 9.6 us against 13.5; not where B is small (64 tokens, 2,560 channels: 5.9
// against 5.6).
constexpr int64_t kLoraNearTiles = 32;         // of 256 channels

// Of these, u by each workgroup itself (FUSED, up to 16 ranks) saves a launch,
// and costs every further workgroup of a compute unit its steps along K, twice
// where K is odd (rows at any byte).  Two launches / one, us in a graph, an
// adapter a token:
//   workgroups a compute unit         1             2            3            4
//   K 2,560 (and 64 to 2,558)     5.6 /  3.8    5.7 /  4.6   5.7 /  5.6   5.9 /  6.4
//   ... rank 8                    5.1 /  3.7    5.3 /  4.4   5.2 /  5.2   5.5 /  5.8
//   K 769, 1,281                  6.7 /  5.0    6.8 /  6.7   6.7 /  8.6
//   K 4,096                       7.0 /  5.2    7.1 /  6.8   7.5 /  8.7
//   ... rank 8                    6.3 /  5.2    6.4 /  6.7
//   K 2,563                       8.7 /  7.0    8.8 / 10.3
//   K 8,192                       9.3 /  7.6    9.4 / 10.0
//   ... rank 8                    8.1 /  7.8    8.2 / 10.2
//   K 7,681                      12.4 / 10.8   12.5 / 17.9
//   ... rank 8                    9.3 / 11.7    9.6 / 19.8
//   K 16,384                     12.3 / 10.8   13.8 / 16.2
// Where the host launches each call, two take 8.0 at least and one 5.8, so what is
// level in a graph is one.
// Values of K that a wave asks for at once, five loads a row: the layer's own
// hidden size in one step.  Steps of 2,048 / of 2,560, one token of rank 16: K 1,024
// 3.5 / 3.8 us, 2,048 3.3 / 3.8, 2,560 4.4 / 3.6, 4,096 4.3 / 5.0, 5,120 5.4 / 4.8,
// 8,192 6.0 / 7.2; steps of 4,096: 4.7 up to 2,560, 4.5 at 4,096.
constexpr int kLoraStep = 2560;

constexpr bool lora_fused(int64_t workgroups, int64_t K, int r)
{
    const int64_t steps = ceil_div(K, kLoraStep) * (K % 2 == 0 ? 1 : 2), further = ceil_div(workgroups, kCus) - 1;
    return r <= 16 && K >= 8 && steps <= (r > 8 ? 8 : 4) && further * steps <= (r > 8 || steps == 1 ? 2 : 0);
}

struct LoraPlan {
    bool few, fused, near;
    int shrink_slots, expand_slots;
};

// The adapters of a tile of 16 tokens are dealt to so many workgroups (at most
// 16: a token each) that there is one for every compute unit (300 tokens of 9
// requests, rank 64: 10.1 us, the whole tile by one 16.6; 512 tokens with an
// adapter each, rank 32: 34.7, 73.2).
constexpr int lora_slots(int64_t tiles, int64_t target)
{
    int slots = 1;
    while (slots < 16 && tiles * slots < target) slots *= 2;
    return slots;
}

constexpr LoraPlan lora_plan(int64_t M, int64_t N, int64_t K, int r)
{
    LoraPlan p{};
    const int64_t tn = ceil_div(N, 256), tm = ceil_div(M, 16);
    p.few = M * lora_padded(r) <= kLoraFewValues && M * r * (K + N) <= kLoraFewReads;
    p.near = tn >= kLoraNearTiles;
    p.fused = p.few && lora_fused(M * tn, K, r);
    p.shrink_slots = lora_slots(tm * ceil_div(r, r > 16 ? 32 : 16), kCus);
    p.expand_slots = lora_slots(tm * tn, 4 * kCus);
    return p;
}

// Rows of the int8 product that are kept in fp32 at a time on the way to bf16:
// 256 MB of them, and 256 at least.
constexpr int64_t lora_product_rows(int64_t N) { return std::max<int64_t>(256, (1ll << 26) / N / 256 * 256); }

}  // namespace moe
