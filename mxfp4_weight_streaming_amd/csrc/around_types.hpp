// around_types.hpp -- argument blocks and limits of the operators around the
// expert layer, shared by their kernels, their launchers and the C ABI.
#pragma once

#include <stdint.h>

namespace moe {

// moe_type and moe_quant and moe_score of the public header.
enum : int { kTypeBf16 = 0, kTypeF32 = 1 };
enum : int { kQuantNone = 0, kQuantE4m3 = 1, kQuantInt8 = 2 };
enum : int { kScoreSoftmax = 0, kScoreSigmoid = 1 };

constexpr int kMaxNormHidden = 32768;   // 512 threads with 8 vectors of 8 elements each hold a row
constexpr int kMaxGroups = 64;          // one lane a group
constexpr int kMaxAlternatives = 32;    // top alternatives of a row of logits
constexpr int64_t kMaxRowStride = 1ll << 30;   // elements between rows of logits
constexpr int kMaxLoraRank = 128;
constexpr int kMaxLoraDepth = 1 << 24;   // (32 rows are addressed with 32 bits)
constexpr int kMaxAdapters = 65535;
constexpr int kMaxInt8Depth = 131071;   // 131071 * 128 * 128 < 2^31

struct NormArgs {
    const void* x;
    const void* residual;      // or nullptr
    const void* weight;
    void* residual_out;        // or nullptr
    uint16_t* y;               // or nullptr
    uint8_t* q;                // or nullptr
    float* scale;
    double eps;
    int64_t M;
    int H, x_type, r_type, w_type, q_type;
};

struct ScoreArgs {
    const float* logits;   // [M,E]
    const float* bias;     // [E] or nullptr
    int32_t* ids;          // [M,K]
    float* w;              // [M,K]
    int64_t M;
    int E, K, score, G, group_topk, group_score, renormalise;
    float factor;
};

struct Int8Args {
    const uint8_t* a;      // [M,K]
    const uint8_t* w;      // [N,K]
    const float* a_scale;  // [M]
    const float* w_scale;  // [N]
    void* out;             // [M,N]
    int64_t M, N;
    int K, out_type;
    int xm;                // tile kernels: parts along the tokens, of 8 (1, 2, 4 or 8)
};

struct RowSums;

struct LogprobArgs {
    const void* logits;      // [M, V], rows `stride` elements apart
    const int32_t* tokens;   // [M] or nullptr
    float* logprob;          // [M] or nullptr
    int32_t* rank;           // [M] or nullptr
    float* entropy;          // [M] or nullptr
    int32_t* topk_ids;       // [M, topk]
    float* topk_logprob;
    void* ws;
    int64_t M, stride;
    int V, type, topk;
    // by the launcher: LogprobPlan, and the workspace's parts
    int segments, group_segments, groups, parts, part_segments;
    float* maxima;           // [M][groups][256 threads]
    RowSums* sums;           // [M][parts]
};

struct LoraArgs {
    const uint16_t* x;       // [M, K]
    const uint16_t* a;       // [L, r, K]
    const uint16_t* b;       // [L, N, r]
    const float* scale;      // [L] or nullptr (1)
    const int32_t* ids;      // [M]
    const void* base;        // [M, N] or nullptr (0)
    void* out;               // [M, N]
    float* u;                // [M, rp], workspace
    int64_t M, N;
    int K, r, rp, L, out_type;   // rp: r up to a multiple of 32
    // by the launcher
    int slots;               // workgroups that share a tile's adapters
    bool near;               // workgroups of the same channels on one XCD
};

}  // namespace moe
