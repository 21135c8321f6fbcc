// score_kernels.hpp -- routing by scores (gfx950): sigmoid or softmax scores,
// balance bias, groups, top-K, weights.
//
//   s = fl32(sigmoid(l)) or fl32(softmax(l)), c = fl32(s + bias)
//   group value = sum of the n largest available c of the group
//   ids = the K largest c in the group_topk best groups; w = s[ids] / sum * factor
//
// The ids are compared for equality by whoever checks a router, and two
// experts' scores may be neighbours in fp32, so the scores are evaluated in
// fp64 and rounded once: any evaluation that accurate gives the same fp32
// values and so the same ids.  From there on everything is exact comparison
// of fp32 keys and fp32 additions of two operands.
#pragma once

#include "around_common.hpp"
#include "moe_types.hpp"
#include "topk_wave.hpp"        // f32_orderable

namespace moe {

constexpr int kScoreSlots = kMaxExperts / kWave;   // experts a lane holds: lane, lane + 64, ...

// One wave a token.
__global__ __launch_bounds__(256) void route_scores_kernel(ScoreArgs a)
{
    __shared__ float c_lds[4][kMaxExperts];
    __shared__ float s_lds[4][kMaxExperts];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    float* cl = c_lds[wv];
    float* sl = s_lds[wv];
    const int each = a.E / a.G;
    const uint32_t gone = f32_orderable(-__builtin_inff());   // an unavailable expert's key; 0 is below every key
    for (int64_t m = (int64_t)blockIdx.x * 4 + wv; m < a.M; m += (int64_t)gridDim.x * 4) {
        const float* l = a.logits + (size_t)m * a.E;
        float x[kScoreSlots];
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kScoreSlots; ++i) {
            const int e = lane + i * kWave;
            float v = e < a.E ? l[e] : -__builtin_inff();
            if (v != v) v = -__builtin_inff();
            x[i] = fminf(v, 3.402823466e+38f);
            top = fmaxf(top, x[i]);
        }
        double ex[kScoreSlots], sum = 1.0;
        if (a.score == kScoreSoftmax) {
            top = wave_max(top);
            double part = 0.0;
#pragma unroll
            for (int i = 0; i < kScoreSlots; ++i) {
                ex[i] = __builtin_isinf(x[i]) ? 0.0 : exp((double)x[i] - (double)top);
                part += ex[i];
            }
            sum = wave_sum_f64(part);
            if (sum == 0.0) sum = 1.0;
        }
#pragma unroll
        for (int i = 0; i < kScoreSlots; ++i) {
            const int e = lane + i * kWave;
            if (e < a.E) {
                const float s = a.score == kScoreSoftmax ? (float)(ex[i] / sum) : (float)(1.0 / (1.0 + exp(-(double)x[i])));
                float c = a.bias != nullptr ? s + a.bias[e] : s;
                const bool out = __builtin_isinf(x[i]) || c != c || c == -__builtin_inff();
                cl[e] = out ? -__builtin_inff() : c;
                sl[e] = out ? 0.0f : s;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // lane g: group g's value, then its rank among the groups
        uint64_t stays = ~0ull;
        if (a.G > a.group_topk) {
            uint32_t key = 0;
            if (lane < a.G) {
                float b1 = -__builtin_inff(), b2 = -__builtin_inff();
                for (int i = 0; i < each; ++i) {
                    const float c = cl[lane * each + i];
                    if (c > b1) { b2 = b1; b1 = c; }
                    else if (c > b2) b2 = c;
                }
                const float v = (a.group_score == 2 && b2 > -__builtin_inff()) ? b1 + b2 : b1;
                key = f32_orderable(v + 0.0f);            // -0 counts as +0
            }
            int rank = 0;
            for (int g = 0; g < a.G; ++g) {
                const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)key, g);
                rank += (other > key || (other == key && g < lane)) ? 1 : 0;
            }
            stays = __ballot(lane < a.G && rank < a.group_topk);
        }
        uint64_t keys[kScoreSlots];
#pragma unroll
        for (int i = 0; i < kScoreSlots; ++i) {
            const int e = lane + i * kWave;
            uint32_t k = 0;
            if (e < a.E && ((stays >> (e / each)) & 1)) k = max(f32_orderable(cl[e] + 0.0f), gone);
            keys[i] = ((uint64_t)k << 32) | (uint32_t)(kMaxExperts - 1 - min(e, kMaxExperts - 1));
        }
        int my_id = 0;
        float my_w = 0.0f, wsum = 0.0f;
        for (int j = 0; j < a.K; ++j) {
            uint64_t best = 0;
#pragma unroll
            for (int i = 0; i < kScoreSlots; ++i) best = max_u64(best, keys[i]);
            best = wave_max_u64(best);
            const int e = kMaxExperts - 1 - (int)(uint32_t)best;
#pragma unroll
            for (int i = 0; i < kScoreSlots; ++i)
                if (keys[i] == best) keys[i] = 0;
            const float w = sl[e];
            wsum += w;
            if (lane == j) {
                my_id = e;
                my_w = w;
            }
        }
        if (a.renormalise) my_w = my_w / (wsum == 0.0f ? 1.0f : wsum);
        if (lane < a.K) {
            a.ids[(size_t)m * a.K + lane] = my_id;
            a.w[(size_t)m * a.K + lane] = my_w * a.factor;
        }
        __builtin_amdgcn_wave_barrier();                  // the next token takes this wave's LDS
    }
}

}  // namespace moe
