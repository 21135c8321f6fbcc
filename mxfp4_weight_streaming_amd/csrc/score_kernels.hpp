// score_kernels.hpp -- routing by scores (gfx950): sigmoid or softmax scores,
// balance bias, groups, top-K, weights.
//
//   s = fl32(sigmoid(l)) or fl32(softmax(l)), c = fl32(s + bias)
//   group value = sum of the n largest available c of the group
//   ids = the K largest c in the group_topk best groups; w = s[ids] / sum * factor
//
// Two experts' scores may be neighbours in fp32, and a choice between them
// should not hang on how a kernel approximates: the scores are evaluated in fp64,
// off by less than 2^-50 of a sigmoid or 2^-46 of a softmax score (its
// exponentials 2^-51, the sum of up to 512 of them 14 roundings, and a logit's
// distance from the largest, up to 104 where it counts, up to 2^-47), and
// rounded once.  Two evaluations that accurate give the same fp32 value unless
// the exact one lies that near the middle between two fp32 numbers: at most one
// score in 2^25, or in 2^21.  From there on everything is exact comparison of fp32
// keys and fp32 additions of two operands.
//
// One wave a token, PER consecutive experts a lane (E <= 64 PER), so that a
// group is a run of lanes and its two largest are found in registers.
//
// Sigmoid scores depend on their own logit alone, so only the few that may be
// chosen are evaluated in fp64: fp32 approximations, off by less than a known
// margin, choose the groups and bound the K-th largest c from below, and the
// experts at or above that bound less the margin, one a lane, get their exact
// scores.  Where the margin leaves the groups open, or the candidates do not
// fit the wave, every score is evaluated exactly.  Softmax scores share the sum
// of all exponentials and are always evaluated exactly.
#pragma once

#include "around_common.hpp"
#include "exp_coefs.hpp"
#include "moe_types.hpp"
#include "topk_wave.hpp"        // f32_orderable

namespace moe {

// e^x for |x| <= 200, relative error below 2^-51: x = n ln2 + r, |r| <= ln2 / 2,
// 1 + r + r^2 q(r) with the constants of exp_coefs.hpp, times 2^n.  What is
// off: q by 2^-55, r by 2^-54 (the two roundings of x - n ln2; ln2 to one
// double only would add 2^-47 at n = 288), the last two steps by 2^-54.5 and
// 2^-53: less than 2^-51.9 in all, 2^-52.4 the most seen
// (tests/exp_f64_check.cpp).  The sum of 1.5 * 2^52 and x / ln2 rounds to a
// whole number in its low word.
// The coefficients are put into scalar registers where they are used: as
// literals each would be copied into vector registers, ahead of the loop over
// the tokens, and stay there.
struct ExpCoefs {
    double c[kExpTerms], ln2_low;
    __device__ __forceinline__ ExpCoefs()
    {
#pragma unroll
        for (int i = 0; i < kExpTerms; ++i) c[i] = kExpQ[i];
        ln2_low = kExpLn2Low;
#pragma unroll
        for (int i = 0; i < kExpTerms - 1; ++i) asm volatile("" : "+s"(c[i]));   // (0.5 needs no register)
        asm volatile("" : "+s"(ln2_low));
    }
};

__device__ __forceinline__ double exp_f64(double x, const ExpCoefs& k)
{
    const double t = __builtin_fma(x, kExpLog2E, 0x1.8p+52);
    const double n = t - 0x1.8p+52;
    const double r = __builtin_fma(-n, k.ln2_low, __builtin_fma(-n, kExpLn2, x));
    double p = k.c[0];
#pragma unroll
    for (int i = 1; i < kExpTerms; ++i) p = __builtin_fma(p, r, k.c[i]);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
}

// 1 / d for d in [1, 2^300]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp_f64(double d)
{
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// fl32(sigmoid(x)); beyond +-200 that is 0 or 1 anyway, and NaN gives 0 or 1.
__device__ __forceinline__ float sigmoid_exact(float x)
{
    const ExpCoefs k;
    return (float)rcp_f64(1.0 + exp_f64(-(double)__builtin_amdgcn_fmed3f(x, -200.0f, 200.0f), k));
}

// The same in fp32, off by less than 2^-20: the product with log2 e is off by
// 2^-24 of itself, which moves sigmoid by at most 0.28 * 2^-24; exp2, the sum
// and the reciprocal by at most 4 * 2^-24 together.
__device__ __forceinline__ float sigmoid_near(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * __builtin_amdgcn_fmed3f(x, -80.0f, 80.0f)));
}

// How far a choice value c made of sigmoid_near may be from the exact one:
// 2^-20, and the roundings of the two sums, 2^-24 |c| each.  Twice that, for
// safety.
__device__ __forceinline__ float near_margin(float c) { return 0x1p-19f + 0x1p-22f * fabsf(c); }

// Choice values are handled as orderable keys: comparisons of unsigned numbers,
// without the care that fp32 minima and maxima take of NaN.  0 is below every
// key; kNoChoice is the key of -inf, an unavailable expert's.
constexpr uint32_t kNoChoice = 0x007FFFFFu;

// The two largest of a set of keys (b1 >= b2).
struct Top2 {
    uint32_t b1, b2;
    __device__ __forceinline__ void take(uint32_t v)
    {
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
    }
    __device__ __forceinline__ void take(const Top2& o)
    {
        b2 = max(min(b1, o.b1), max(b2, o.b2));
        b1 = max(b1, o.b1);
    }
};

template <int CTRL>
__device__ __forceinline__ void merge_dpp(Top2& t)
{
    const Top2 o = {dpp_u32<CTRL>(t.b1), dpp_u32<CTRL>(t.b2)};
    t.take(o);
}

constexpr int kDppRowRor8 = 0x128;    // rotation of a row by 8: lane ^ 8

// The value of lane ^ 16 or lane ^ 32 beside a lane's own, in either order:
// what is taken of both must not depend on it.
struct Both {
    uint32_t a, b;
};

template <int MASK>
__device__ __forceinline__ Both lane_pair(uint32_t v)
{
    static_assert(MASK == 16 || MASK == 32, "rows of 16 or halves of 32 lanes");
    if constexpr (MASK == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return Both{(uint32_t)r[0], (uint32_t)r[1]};
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return Both{(uint32_t)r[0], (uint32_t)r[1]};
    }
}

template <int MASK>
__device__ __forceinline__ void merge_pair(Top2& t)
{
    const Both b1 = lane_pair<MASK>(t.b1), b2 = lane_pair<MASK>(t.b2);
    t = Top2{b1.a, b2.a};
    t.take(Top2{b1.b, b2.b});
}

// Merge over aligned runs of `lanes` lanes, a power of two.
__device__ __forceinline__ void merge_lanes(Top2& t, int lanes)
{
    if (lanes >= 2) merge_dpp<kDppXor1>(t);
    if (lanes >= 4) merge_dpp<kDppXor2>(t);
    if (lanes >= 8) merge_dpp<kDppHalfMirror>(t);
    if (lanes >= 16) merge_dpp<kDppMirror>(t);
    if (lanes >= 32) merge_pair<16>(t);
    if (lanes >= 64) merge_pair<32>(t);
}

// A candidate: what its exact score and choice value are made of.
struct Candidate {
    float logit, bias;
    int32_t expert, unused;
};

// A wave's LDS: the candidates and their keys; or all choice values, where the
// groups are no runs of lanes.
struct ScoreLds {
    union {
        struct {
            Candidate cand[kWave];
            uint64_t key[kWave];
        };
        uint32_t choice[kMaxExperts];
    };
};

__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16,384 tokens over 512 experts, sigmoid, 4 of 8 groups: 24-25 us (1.4 TB/s of
// logits); over 256, softmax: 15 us; one token 4.4 us in a graph.  Bound by the
// issue of vector instructions (613 a token at 512 experts, in issue 85% of the
// time; 427 and 92% at 256, softmax), not by the logits' bytes (7 and 3 us).
// Every score in fp64 took half as many again and 31 us; the first kernel, with
// groups and choice through LDS, 57 us.  Holding the next token's logits in registers gained nothing: it cost
// waves.
template <int PER, bool SOFTMAX>
__global__ __launch_bounds__(256) void route_scores_kernel(ScoreArgs a)
{
    __shared__ __attribute__((aligned(16))) ScoreLds lds_all[4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    ScoreLds& lds = lds_all[wv];
    const int E = a.E, K = a.K, G = a.G, each = E / G;
    int e0 = lane * PER;
    const int group0 = e0 / each, left0 = each - (e0 - group0 * each);
    const float none = -__builtin_inff();
    typedef uint32_t vec_t __attribute__((ext_vector_type(PER), aligned(4)));
    auto load = [&](const float* p, float (&v)[PER]) {     // this lane's experts of one row
        if (e0 + PER <= E) {
            const vec_t r = *reinterpret_cast<const vec_t*>(p + e0);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if constexpr (PER == 1) v[i] = __uint_as_float((uint32_t)r[0]);
                else v[i] = __uint_as_float(r[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = e0 + i < E ? p[e0 + i] : none;
        }
    };
    float bias[PER] = {};                                  // no bias: + 0 changes no score
    if (a.bias != nullptr) {
        load(a.bias, bias);
#pragma unroll
        for (int i = 0; i < PER; ++i) bias[i] = fmaxf(bias[i], none);   // NaN as -inf
    }
    const int64_t stride = (int64_t)gridDim.x * 4;
    int64_t m = (int64_t)blockIdx.x * 4 + wv;
    for (; m < a.M; m += stride) {
        asm volatile("" : "+v"(e0));                       // or every e0 + i stays in a register over all tokens
        float x[PER];
        load(a.logits + (size_t)m * E, x);
        // softmax: the largest logit, and 1 / the sum of exponentials
        float top = none;
        double inv = 0.0;
        if constexpr (SOFTMAX) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                x[i] = fminf(fmaxf(x[i], none), 3.402823466e+38f);   // NaN as -inf
                top = fmaxf(top, x[i]);
            }
            top = wave_max(top);
        }
        auto part = [&](float logit, const ExpCoefs& k) {
            return logit > none ? exp_f64(fmax((double)logit - (double)top, -200.0), k) : 0.0;
        };
        auto score_exact = [&](float logit) {
            return SOFTMAX ? (float)(part(logit, ExpCoefs()) * inv) : sigmoid_exact(logit);
        };
        // the choice value's key; kNoChoice where the logit is -inf or NaN or
        // the bias -inf.  The value is never -0: a score is at least +0.
        auto choice = [&](float logit, float score, float b) {
            const uint32_t u = __float_as_uint(score + b);
            return logit > none ? u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u) : kNoChoice;
        };
        int rank = kWave, id = 0;
        float w = 0.0f;
        for (bool exact = SOFTMAX;; exact = true) {
            uint32_t key[PER];
            if constexpr (SOFTMAX) {
                const ExpCoefs k;
                double ex[PER], sum = 0.0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    ex[i] = part(x[i], k);
                    sum += ex[i];
                }
                sum = wave_sum_f64(sum);
                inv = sum > 0.0 ? rcp_f64(sum) : 0.0;
#pragma unroll
                for (int i = 0; i < PER; ++i) key[i] = choice(x[i], (float)(ex[i] * inv), bias[i]);
            } else if (exact) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    float l = x[i];
                    asm volatile("" : "+v"(l));            // else computed for every token, ahead of the branch
                    key[i] = choice(l, sigmoid_exact(l), bias[i]);
                    __builtin_amdgcn_sched_barrier(0);     // one at a time: the path is rare, its registers are not
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) key[i] = choice(x[i], sigmoid_near(x[i]), bias[i]);
            }
            if (E < PER * kWave) {                         // experts past E: out of the running
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (e0 + i >= E) key[i] = 0;
            }
            uint32_t best = 0;                             // the lane's largest key in the groups that stay
#pragma unroll
            for (int i = 0; i < PER; ++i) best = max(best, key[i]);
            bool lane_stays = true;
            if (G > a.group_topk) {
                // a group's value, of its two largest keys
                auto value = [&](const Top2& t) {
                    const float v = f32_from_orderable(t.b1);
                    return a.group_score == 2 && t.b2 > kNoChoice ? v + f32_from_orderable(t.b2) : v;
                };
                // rank of a group among all, whose keys stand in lanes 0, step, 2 step, ...
                auto rank_of = [&](uint32_t group_key, int step, int mine) {
                    int r = 0;
                    for (int g = 0; g < G; ++g) {
                        const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)group_key, g * step);
                        r += (other > group_key || (other == group_key && g < mine)) ? 1 : 0;
                    }
                    return r;
                };
                // near values: whether any group that goes may, within the
                // errors of its two summands, be worth as much as one that stays
                auto open = [&](const Top2& t, bool group, bool stay) {
                    const float v = value(t), c2 = t.b2 > kNoChoice ? f32_from_orderable(t.b2) : 0.0f;
                    float e = 2.0f * near_margin(fabsf(f32_from_orderable(t.b1)) + fabsf(c2));
                    if (!(e < 0x1p127f)) e = 0.0f;         // no available expert, or +inf: exact
                    const float last = f32_from_orderable(wave_min_u32(group && stay ? f32_orderable(v - e) : 0xFFFFFFFFu));
                    const float first = f32_from_orderable(wave_max_u32(group && !stay ? f32_orderable(v + e) : 0u));
                    return !(last > first);
                };
                const int run = each / PER;
                bool unclear = false;
                if (each % PER == 0 && (run & (run - 1)) == 0) {
                    Top2 t = {kNoChoice, kNoChoice};
#pragma unroll
                    for (int i = 0; i < PER; ++i) t.take(key[i]);
                    merge_lanes(t, run);
                    const uint32_t group_key = f32_orderable(value(t));
                    lane_stays = rank_of(group_key, run, lane / run) < a.group_topk;
                    if (!exact) unclear = open(t, e0 < E, lane_stays);
                    if (!lane_stays) best = 0;
                } else {                                   // lane g: group g, from LDS
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (e0 + i < E) lds.choice[e0 + i] = key[i];
                    wave_lds_fence();
                    Top2 t = {kNoChoice, kNoChoice};
                    if (lane < G)
                        for (int i = 0; i < each; ++i) t.take(lds.choice[lane * each + i]);
                    const uint32_t group_key = f32_orderable(value(t));
                    const bool stay = rank_of(group_key, 1, lane) < a.group_topk;
                    if (!exact) unclear = open(t, lane < G, stay);
                    const uint64_t kept = __ballot(lane < G && stay);
                    best = 0;
                    int group = group0, left = left0;      // expert e0 + i: its group, and experts to the next
                    asm volatile("" : "+v"(group));        // kept in this branch
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        if (!((kept >> min(group, kMaxGroups - 1)) & 1)) key[i] = 0;   // (past E: 0 already)
                        best = max(best, key[i]);
                        if (--left == 0) {
                            left = each;
                            ++group;
                        }
                    }
                    wave_lds_fence();                      // the candidates take the LDS
                }
                if (unclear) continue;
            }
            // Threshold: the largest key of each of 8 sets of lanes (l mod 8,
            // so that every group has lanes in every set) are 8 different
            // entries, so the K <= 8 largest are at or above the smallest of the
            // 8, less the margin of both.  The entries there, mostly few, are
            // ranked by counting.
            const Both far = lane_pair<32>(best);
            const Both near = lane_pair<16>(max(far.a, far.b));
            best = max(near.a, near.b);
            best = max(best, dpp_u32<kDppRowRor8>(best));
            best = min(best, dpp_u32<kDppXor1>(best));
            best = min(best, dpp_u32<kDppXor2>(best));
            best = min(best, dpp_u32<kDppHalfMirror>(best));
            uint32_t thr = max((uint32_t)__builtin_amdgcn_readlane((int)best, 0), 1u);
            if (!exact && thr > kNoChoice && thr < 0xFF800000u) {   // finite
                const float v = f32_from_orderable(thr);
                thr = f32_orderable(v - 2.0f * near_margin(v));
            }
            if (!lane_stays) thr = 0xFFFFFFFFu;            // above every key
            uint64_t hit[PER];
            int nc = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                hit[i] = __ballot(key[i] >= thr);
                nc += __popcll(hit[i]);
            }
            if (nc > kWave) {                              // many equal keys: K rounds of the largest
                if (!exact) continue;
                Candidate me = {none, 0.0f, 0, 0};
                for (int j = 0; j < K; ++j) {
                    uint64_t most = 0;
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (lane_stays) most = max_u64(most, ((uint64_t)key[i] << 32) | (uint32_t)(0xFFFF - (e0 + i)));
                    most = wave_max_u64(most);
                    const int e = 0xFFFF - (int)(uint32_t)(most & 0xFFFFu);
                    float l = 0.0f, b = 0.0f;
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (e == e0 + i) {
                            l = x[i];
                            b = bias[i];
                            key[i] = 0;
                        }
                    l = row_lane(l, e / PER);
                    b = row_lane(b, e / PER);
                    if (lane == j) {
                        me = Candidate{l, b, e, 0};
                        rank = j;
                    }
                }
                if (rank < K) {
                    id = me.expert;
                    w = score_exact(me.logit);
                    if (choice(me.logit, w, me.bias) <= kNoChoice) w = 0.0f;
                }
                break;
            }
            int base = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (key[i] >= thr) {
                    const int pos = base + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(hit[i] >> 32),
                                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)hit[i], 0u));
                    lds.cand[pos] = Candidate{x[i], bias[i], e0 + i, 0};
                }
                base += __popcll(hit[i]);
            }
            wave_lds_fence();
            const Candidate me = lds.cand[lane];           // (behind the last: not used)
            const float score = score_exact(me.logit);
            const uint32_t value = choice(me.logit, score, me.bias);
            const uint64_t mine = lane < nc ? ((uint64_t)value << 32) | (uint32_t)(0xFFFF - me.expert) : 0;
            lds.key[lane] = mine;
            wave_lds_fence();
            int above = 0;
            for (int j = 0; j < nc; j += 8) {              // broadcast reads, 8 keys a round trip
                ulonglong2 kk[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) kk[q] = *reinterpret_cast<const ulonglong2*>(lds.key + j + 2 * q);
#pragma unroll
                for (int q = 0; q < 4; ++q) above += (kk[q].x > mine ? 1 : 0) + (kk[q].y > mine ? 1 : 0);
            }
            if (lane < nc) {
                rank = above;
                id = me.expert;
                w = rank < K && value > kNoChoice ? score : 0.0f;
            }
            wave_lds_fence();                              // the next token takes the LDS
            break;
        }
        if (a.renormalise) {
            const float sum = wave_sum(w);
            w = w / (sum == 0.0f ? 1.0f : sum);
        }
        if (rank < K) {
            a.ids[(size_t)m * K + rank] = id;
            a.w[(size_t)m * K + rank] = w * a.factor;
        }
    }
}

}  // namespace moe
