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
#include "moe_types.hpp"
#include "topk_wave.hpp"        // f32_orderable

namespace moe {

// e^x for |x| <= 200, relative error below 2^-45: x = n ln2 + r, |r| <= ln2 / 2,
// the Taylor sum of e^r to r^11 / 11! (the next term is below 2^-47), times 2^n.
// The sum of 1.5 * 2^52 and x / ln2 rounds to a whole number in its low word.
// The coefficients are kept in scalar registers: as literals each product would
// first copy one into a vector register.
struct ExpCoefs {
    double c[10];
    __device__ __forceinline__ ExpCoefs()
    {
        c[0] = 1.0 / 39916800.0;
        c[1] = 1.0 / 3628800.0;
        c[2] = 1.0 / 362880.0;
        c[3] = 1.0 / 40320.0;
        c[4] = 1.0 / 5040.0;
        c[5] = 1.0 / 720.0;
        c[6] = 1.0 / 120.0;
        c[7] = 1.0 / 24.0;
        c[8] = 1.0 / 6.0;
        c[9] = 0.5;
#pragma unroll
        for (int i = 0; i < 9; ++i) asm volatile("" : "+s"(c[i]));
    }
};

__device__ __forceinline__ double exp_f64(double x, const ExpCoefs& k)
{
    const double t = __builtin_fma(x, 0x1.71547652b82fep+0, 0x1.8p+52);
    const double n = t - 0x1.8p+52;
    const double r = __builtin_fma(-n, 0x1.62e42fefa39efp-1, x);
    double p = k.c[0];
#pragma unroll
    for (int i = 1; i < 10; ++i) p = __builtin_fma(p, r, k.c[i]);
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
__device__ __forceinline__ float sigmoid_exact(float x, const ExpCoefs& k)
{
    return (float)rcp_f64(1.0 + exp_f64(-(double)__builtin_amdgcn_fmed3f(x, -200.0f, 200.0f), k));
}

// The same in fp32, off by less than 2^-20: the product with log2 e is off by
// 2^-24 of itself, which moves sigmoid by at most 0.28 * 2^-24; exp2, the sum
// and the reciprocal by at most 4 * 2^-24 together.
__device__ __forceinline__ float sigmoid_near(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * __builtin_amdgcn_fmed3f(x, -80.0f, 80.0f)));
}

// How far a choice value made of sigmoid_near may be from the exact one:
// 2^-20, and the two sums' roundings.  Twice that, for safety.
__device__ __forceinline__ float near_margin(float c) { return 0x1p-19f + 0x1p-22f * fabsf(c); }

// The two largest of a set of values (b1 >= b2); -inf where there is none.
struct Top2 {
    float b1, b2;
    __device__ __forceinline__ void take(float v)
    {
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
    }
    __device__ __forceinline__ void take(const Top2& o)
    {
        b2 = fmaxf(fminf(b1, o.b1), fmaxf(b2, o.b2));
        b1 = fmaxf(b1, o.b1);
    }
};

template <int CTRL>
__device__ __forceinline__ void merge_dpp(Top2& t)
{
    const Top2 o = {dpp_f32<CTRL>(t.b1), dpp_f32<CTRL>(t.b2)};
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
    const Both b1 = lane_pair<MASK>(__float_as_uint(t.b1)), b2 = lane_pair<MASK>(__float_as_uint(t.b2));
    t = Top2{__uint_as_float(b1.a), __uint_as_float(b2.a)};
    t.take(Top2{__uint_as_float(b1.b), __uint_as_float(b2.b)});
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
        float c[kMaxExperts];
    };
};

__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16,384 tokens over 512 experts, sigmoid, 4 of 8 groups: 29 us (1.2 TB/s of
// logits); over 256, softmax: 17 us; one token 4.9 us in a graph.  Bound by the
// issue of ~500 instructions a token and the chain of reductions between them,
// not by the logits' bytes (7 us).  Every score in fp64 took 31 us and 871
// instructions; the first kernel, with groups and choice through LDS, 57 us.
// Bounding the registers for 4 waves a SIMD instead of 3 spills and gains
// nothing.
template <int PER, bool SOFTMAX>
__global__ __launch_bounds__(256) void route_scores_kernel(ScoreArgs a)
{
    __shared__ __attribute__((aligned(16))) ScoreLds lds_all[4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    ScoreLds& lds = lds_all[wv];
    const int E = a.E, K = a.K, G = a.G, each = E / G, e0 = lane * PER;
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
    float bias[PER] = {};
    if (a.bias != nullptr) load(a.bias, bias);
    const ExpCoefs k;
    const int64_t stride = (int64_t)gridDim.x * 4;
    int64_t m = (int64_t)blockIdx.x * 4 + wv;
    if (m >= a.M) return;
    float ahead[PER];                                      // the next token's logits
    load(a.logits + (size_t)m * E, ahead);
    for (; m < a.M; m += stride) {
        float x[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = ahead[i];
        if (m + stride < a.M) load(a.logits + (size_t)(m + stride) * E, ahead);
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
        auto part = [&](float logit) { return logit > none ? exp_f64(fmax((double)logit - (double)top, -200.0), k) : 0.0; };
        auto score_exact = [&](float logit) {
            return SOFTMAX ? (float)(part(logit) * inv) : sigmoid_exact(logit, k);
        };
        // the choice value; -inf where the logit or the value is -inf or NaN.
        // It is never -0: a score is at least +0.
        auto choice = [&](float logit, float score, float b) {
            const float v = a.bias != nullptr ? score + b : score;
            return logit > none ? fmaxf(v, none) : none;
        };
        int rank = kWave, id = 0;
        float w = 0.0f;
        for (bool exact = SOFTMAX;; exact = true) {
            float c[PER];
            if constexpr (SOFTMAX) {
                double ex[PER], sum = 0.0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    ex[i] = part(x[i]);
                    sum += ex[i];
                }
                sum = wave_sum_f64(sum);
                inv = sum > 0.0 ? rcp_f64(sum) : 0.0;
#pragma unroll
                for (int i = 0; i < PER; ++i) c[i] = choice(x[i], (float)(ex[i] * inv), bias[i]);
            } else if (exact) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    float l = x[i];
                    asm volatile("" : "+v"(l));            // else computed for every token, ahead of the branch
                    c[i] = choice(l, sigmoid_exact(l, k), bias[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) c[i] = choice(x[i], sigmoid_near(x[i]), bias[i]);
            }
            // the groups that stay
            bool stays[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) stays[i] = e0 + i < E;
            if (G > a.group_topk) {
                auto value = [&](const Top2& t) { return a.group_score == 2 && t.b2 > none ? t.b1 + t.b2 : t.b1; };
                // rank of a group among all, whose keys stand in lanes 0, step, 2 step, ...
                auto rank_of = [&](uint32_t key, int step, int mine) {
                    int r = 0;
                    for (int g = 0; g < G; ++g) {
                        const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)key, g * step);
                        r += (other > key || (other == key && g < mine)) ? 1 : 0;
                    }
                    return r;
                };
                // near values: whether the last group that stays and the first
                // that goes are too close to tell (a value is a sum of two)
                auto open = [&](float v, bool group, bool stay) {
                    const float last = -wave_max(group && stay ? -v : none), first = wave_max(group && !stay ? v : none);
                    return !(last - first > 4.0f * near_margin(fmaxf(fabsf(last), fabsf(first))));
                };
                const int run = each / PER;
                bool unclear = false;
                if (each % PER == 0 && (run & (run - 1)) == 0) {
                    Top2 t = {none, none};
#pragma unroll
                    for (int i = 0; i < PER; ++i) t.take(c[i]);
                    merge_lanes(t, run);
                    const float v = value(t);
                    const bool stay = rank_of(f32_orderable(v), run, lane / run) < a.group_topk;
                    if (!exact) unclear = open(v, e0 < E, stay);
#pragma unroll
                    for (int i = 0; i < PER; ++i) stays[i] = stays[i] && stay;
                } else {                                   // lane g: group g, from LDS
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (e0 + i < E) lds.c[e0 + i] = c[i];
                    wave_lds_fence();
                    Top2 t = {none, none};
                    if (lane < G)
                        for (int i = 0; i < each; ++i) t.take(lds.c[lane * each + i]);
                    const float v = value(t);
                    const bool stay = rank_of(f32_orderable(v), 1, lane) < a.group_topk;
                    if (!exact) unclear = open(v, lane < G, stay);
                    const uint64_t kept = __ballot(lane < G && stay);
#pragma unroll
                    for (int i = 0; i < PER; ++i) stays[i] = stays[i] && ((kept >> (min(e0 + i, E - 1) / each)) & 1);
                    wave_lds_fence();                      // the candidates take the LDS
                }
                if (unclear) continue;
            }
            // keys: 0 for what is out of the running, below every other; an
            // unavailable expert's is that of -inf
            uint32_t key[PER], best = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                key[i] = stays[i] ? f32_orderable(c[i]) : 0u;
                best = max(best, key[i]);
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
            if (!exact && thr > f32_orderable(none)) {
                const float v = f32_from_orderable(thr);
                thr = f32_orderable(v - 2.0f * near_margin(v));
            }
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
                        most = max_u64(most, ((uint64_t)key[i] << 32) | (uint32_t)(0xFFFF - (e0 + i)));
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
                    if (!(choice(me.logit, w, me.bias) > none)) w = 0.0f;
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
            const float score = score_exact(me.logit), value = choice(me.logit, score, me.bias);
            const uint64_t mine = lane < nc ? ((uint64_t)f32_orderable(value) << 32) | (uint32_t)(0xFFFF - me.expert) : 0;
            lds.key[lane] = mine;
            wave_lds_fence();
            int above = 0;
            for (int j = 0; j < nc; j += 16) {             // broadcast reads, 16 keys a round trip
                ulonglong2 kk[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) kk[q] = *reinterpret_cast<const ulonglong2*>(lds.key + j + 2 * q);
#pragma unroll
                for (int q = 0; q < 8; ++q) above += (kk[q].x > mine ? 1 : 0) + (kk[q].y > mine ? 1 : 0);
            }
            if (lane < nc) {
                rank = above;
                id = me.expert;
                w = rank < K && value > none ? score : 0.0f;
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
