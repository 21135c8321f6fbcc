// logprob_kernels.hpp -- log probabilities of given tokens, with rank, entropy
// and top alternatives (gfx950).
//
// Of a row of logits l (NaN as -inf, +inf as the largest finite fp32), with
// m = max l, S = sum exp(l - m) and T = sum exp(l - m) (l - m):
//   log p(v) = (l_v - m) - log S,   entropy = -sum p log p = log S - T / S,
//   rank(t)  = how many v have l_v > l_t, or l_v = l_t and v < t.
//
// One pass over the row.  A wave takes 1,024 logits at a time (16 a lane) and
// keeps the largest so far and the sums at that reference; they are brought to
// a new one where a larger logit comes, on average H_n times in n such
// segments.  The largest logit's own 1 is kept out of the sum: in a confident
// row log S = log1p(S - 1) is what the others are beside it, which fp32 would
// lose.  A segment's 16 terms a lane are added in fp32, segments in fp64.
//
// The alternatives take no second pass: of every 16 logits of a lane (a group)
// the largest is kept, and the K-th largest of 64 disjoint sets' maxima bounds
// the K-th largest logit from below.  Only groups that reach the bound (24 for
// K = 20 on average, 44 for K = 32) are read again, and what reaches it in them
// is ranked by counting.  Where more than a list's worth reach the bound, many
// logits share its value: larger ones are ranked alike, and the first that equal
// it are found from the row's start (64 rows of 157,184 fp32, all but a few at a
// finite value, 20 alternatives: 40 us, and 37 of flat rows, where such rows
// masked by -inf take 18; a pass for each alternative took 1,300).
//
// What bounds it: many long rows of fp32 the reads (2,048 of 157,184 with 5
// alternatives 251 us, 5.1 TB/s; a second pass alone would cost as much again),
// of bf16 the vector instructions more than anything else (159 us, 4.0 TB/s: 16
// logits of a lane are some 190 of them, 16 of these exponentials, and take two
// thirds of the issue slots, at three waves a SIMD); few rows and short ones
// chains of latencies: one row of 157,184 is a launch, 3.3 us for its parts, a
// launch and 3 us to join them.
#pragma once

#include <type_traits>

#include "around_common.hpp"
#include "beside_choice.hpp"

namespace moe {

constexpr int kLogprobGroupList = 256;      // groups read again
constexpr int kLogprobCandidates = 512;     // logits ranked
constexpr int kLogprobShortList = 128;      // ... of a row that one wave holds

constexpr float kLog2e = 1.44269504f;
constexpr float kLargestLogit = 3.40282347e38f;

// A logit's value as the definitions count it.
__device__ __forceinline__ float logit_value(float x)
{
    return __builtin_fminf(__builtin_fmaxf(__builtin_canonicalizef(x), -__builtin_inff()), kLargestLogit);
}

__device__ __forceinline__ float logit_at(const void* logits, bool f32, size_t i)
{
    return logit_value(load_typed(logits, f32 ? kTypeF32 : kTypeBf16, i));
}

// Whether (x, i) stands before (y, j): larger, or equal with a lower index.
__device__ __forceinline__ bool logit_before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

// The sums of a part of a row at the reference m, its largest logit: s = sum
// e^(l - m) without the `top` logits that equal m, t = sum e^(l - m) (l - m).
// `ahead`: how many stand before the given token.
struct RowSums {
    double s, t;
    float m;
    int32_t top, ahead, pad;
};

__device__ __forceinline__ int wave_sum_i32(int v)
{
    v += (int)dpp_u32<kDppXor1>((uint32_t)v);
    v += (int)dpp_u32<kDppXor2>((uint32_t)v);
    v += (int)dpp_u32<kDppHalfMirror>((uint32_t)v);
    v += (int)dpp_u32<kDppMirror>((uint32_t)v);
    return (__builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16)) +
           (__builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48));
}

// The sums of all lanes' parts (a lane without one: m = -inf and zeros).
__device__ __forceinline__ RowSums join_sums(RowSums a)
{
    const float m = wave_max(a.m);
    double s = 0.0, t = 0.0;
    int top = 0;
    if (a.m == m) {
        s = a.s;
        t = a.t;
        top = a.top;
    } else if (a.m > -__builtin_inff()) {
        const double d = (double)a.m - (double)m, f = exp(d), all = a.s + (double)a.top;
        s = all * f;
        t = (a.t + all * d) * f;
    }
    return RowSums{wave_sum_f64(s), wave_sum_f64(t), m, wave_sum_i32(top), wave_sum_i32(a.ahead), 0};
}

// 16 logits of a lane: vectors of 16 bytes, 64 lanes apart.
template <bool F32>
struct Logits16 {
    static constexpr int kVec = F32 ? 4 : 8, kVecs = 16 / kVec;
    u32x4 v[kVecs];
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (F32) return __uint_as_float(v[i >> 2][i & 3]);
        const uint32_t d = v[i >> 3][(i & 7) >> 1];
        return __uint_as_float(i & 1 ? d & 0xFFFF0000u : d << 16);
    }
    __device__ __forceinline__ void set(int i, float x)   // (of the logits' type)
    {
        const uint32_t d = v[i / kVec][F32 ? i & 3 : (i & 7) >> 1], n = __float_as_uint(x);
        v[i / kVec][F32 ? i & 3 : (i & 7) >> 1] = F32 ? n : i & 1 ? (d & 0xFFFFu) | (n & 0xFFFF0000u) : (d & 0xFFFF0000u) | n >> 16;
    }
    __device__ __forceinline__ void clear(int i) { set(i, -__builtin_inff()); }
};

// 16 bytes less the first `bits` (0 to 128, whole values).
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int bits)
{
    const uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
    const int by = bits & 63;
    const uint64_t a = bits >= 64 ? hi : lo, b = bits >= 64 ? 0 : hi;
    const uint64_t x = by == 0 ? a : a >> by | b << (64 - by), y = b >> by;
    return u32x4{(uint32_t)x, (uint32_t)(x >> 32), (uint32_t)y, (uint32_t)(y >> 32)};
}

typedef uint32_t u32x4_at __attribute__((ext_vector_type(4), aligned(2)));   // at any element

// Element i (0..15) of lane `lane`, in the wave's 1,024.
template <bool F32>
__device__ __forceinline__ int logit_place(int lane, int i)
{
    constexpr int E = Logits16<F32>::kVec;
    return (i / E) * (64 * E) + lane * E + i % E;
}

// The given token of a row, and its logit.
struct Asked {
    int token;                                           // (-1 where the call asks for none)
    float mine;
    bool inside;                                         // 0 <= token < V
};

template <bool F32>
__device__ __forceinline__ Asked asked_of(const LogprobArgs& g, int64_t m, const uint8_t* row)
{
    Asked a;
    a.token = g.tokens != nullptr ? g.tokens[m] : -1;
    a.inside = a.token >= 0 && a.token < g.V;
    a.mine = a.inside ? logit_at(row, F32, (size_t)a.token) : 0.0f;
    return a;
}

template <bool F32>
__device__ __forceinline__ const uint8_t* row_of(const LogprobArgs& g, int64_t m)
{
    return static_cast<const uint8_t*>(g.logits) + (size_t)m * (size_t)g.stride * (F32 ? 4 : 2);
}

// A wave's walk over its segments of one row's part.
template <bool F32>
struct LogitWalk {
    const uint8_t* row;
    int V, lane;
    // the given token, if its rank is asked for
    int token;
    bool asked;
    float mine, above;                                   // its logit, and the next larger number
    // state: s = sum 2^z and t = sum 2^z z a lane, with z = log2(e) l - ref; the
    // rest the wave's: m its largest, `top` logits equal to it and not in s
    double s = 0.0, t = 0.0;
    float m = -__builtin_inff(), ref = 0.0f;
    int top = 0, ahead = 0;

    // log2(e) m - ref, which is 0 but for ref's rounding
    __device__ __forceinline__ double off() const { return (double)m * (double)kLog2e - (double)ref; }

    // Brings the sums to a new reference; d = the old one less the new one.
    __device__ __forceinline__ void rebase(double d)
    {
        if (s != 0.0) {                                  // (d may be infinite, and a NaN where s is 0)
            const double f = exp(d * 0.69314718055994531);
            t = f == 0.0 ? 0.0 : (t + s * d) * f;
            s *= f;
        }
    }

    __device__ __forceinline__ void load(int at, Logits16<F32>& x) const
    {
        constexpr int E = Logits16<F32>::kVec, B = F32 ? 4 : 2;
        if (at + 1024 <= V) {
#pragma unroll
            for (int u = 0; u < Logits16<F32>::kVecs; ++u)
                x.v[u] = *reinterpret_cast<const u32x4_at*>(row + (size_t)(at + (u * 64 + lane) * E) * B);
            return;
        }
        // The row's end: a vector that would pass it is the row's last one, shifted
        // down, with -inf behind; all are asked for before one is waited for.
        if (V >= E) {
#pragma unroll
            for (int u = 0; u < Logits16<F32>::kVecs; ++u)
                x.v[u] = *reinterpret_cast<const u32x4_at*>(row + (size_t)min(at + (u * 64 + lane) * E, V - E) * B);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < Logits16<F32>::kVecs; ++u) {
                const int p = at + (u * 64 + lane) * E;
                if (at + u * 64 * E < V) {
                    x.v[u] = shift_down(x.v[u], min(max(p - (V - E), 0), E) * 8 * B);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (p + e >= V) x.clear(u * E + e);
                } else {
                    x.v[u] = F32 ? u32x4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u}
                                 : u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int p = at + (i / E * 64 + lane) * E + i % E;
                x.clear(i);
                if (p < V) x.set(i, load_typed(row, F32 ? kTypeF32 : kTypeBf16, p));
            }
        }
    }

    // Adds the 1,024 logits from `at`; returns the lane's largest.  Exponentials
    // and the sums of 16 are fp32, some 80 of 190 instructions as it is: a term at
    // a distance d from the largest is off by 2^-24 (2.5 |d| + 24) of itself, which
    // is what log S is allowed.  The logits stay as they are: the maxima pass over
    // NaN, which the clamp of a distance takes to e^-256 = 0 as it does -inf; an
    // infinite one is put right where it is met as the largest.
    __device__ __forceinline__ float add(int at, const Logits16<F32>& raw)
    {
        const float inf = __builtin_inff();
        if (at >= V) return -inf;
        float x[16];
        float largest = -inf;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_canonicalizef(raw.get(i));  // (a signalling NaN would end a chain of v_max3)
            largest = fmaxf(largest, x[i]);
        }
        bool equal = false;                              // whether a logit may equal m
        if (__any(largest >= m)) {
            float most = wave_max(largest);
            if (most == inf) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = x[i] == inf ? kLargestLogit : x[i];
                largest = fminf(largest, kLargestLogit);
                most = kLargestLogit;
            }
            if (most > m) {
                // (never -inf itself: z of -inf would be +inf)
                const float to = fmaxf(most * kLog2e, -kLargestLogit);
                if (m > -inf) {
                    const float z = (float)off(), e = __builtin_amdgcn_exp2f(z);
                    if (lane == 0 && e != 0.0f) {
                        s += (double)top * (double)e;
                        t += (double)top * (double)e * (double)z;
                    }
                    rebase((double)ref - (double)to);
                }
                m = most;
                ref = to;
                top = 0;
            }
            equal = true;
        }
        if (m > -inf) {                                  // (else nothing yet)
            float ss[4] = {0.0f, 0.0f, 0.0f, 0.0f}, tt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            auto sums = [&](auto exclude) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float z = fmaxf(fmaf(x[i], kLog2e, -ref), -256.0f);
                    float e = __builtin_amdgcn_exp2f(z);
                    if constexpr (decltype(exclude)::value) {
                        top += __popcll(__ballot(x[i] == m));
                        e = x[i] == m ? 0.0f : e;
                    }
                    ss[i & 3] += e;
                    tt[i & 3] = fmaf(e, z, tt[i & 3]);
                }
            };
            if (equal) sums(std::true_type{});
            else sums(std::false_type{});
            s += (double)((ss[0] + ss[1]) + (ss[2] + ss[3]));
            t += (double)((tt[0] + tt[1]) + (tt[2] + tt[3]));
        }
        if (asked) {
            if (at + 1024 <= token && mine == -inf) {
                ahead += 1024;                           // all are equal or larger
            } else if (at + 1024 <= V && (at + 1024 <= token || token < at)) {
                // before the token equal logits count, behind it only larger ones
                const float bar = token < at ? above : mine;
                int below = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) below += __popcll(__ballot(!(x[i] >= bar)));
                ahead += 1024 - below;
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    constexpr int E = Logits16<F32>::kVec;
                    if (at + i / E * (64 * E) >= V) break;
                    const int p = at + logit_place<F32>(lane, i);
                    ahead += __popcll(__ballot(p < V && logit_before(logit_value(x[i]), p, mine, token)));
                }
            }
        }
        return largest;
    }

    // The wave's sums at the reference m, in natural logarithms.
    __device__ __forceinline__ RowSums sums()
    {
        s = wave_sum_f64(s);
        t = wave_sum_f64(t);
        rebase(-off());
        return RowSums{s, t * 0.69314718055994531, m, top, ahead, 0};
    }
};

// Order of floats (no NaN) as unsigned numbers, and back.
__device__ __forceinline__ uint32_t float_order(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);        // (+ 0: no -0)
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float order_float(uint32_t o)
{
    return __uint_as_float(o ^ ((int32_t)o < 0 ? 0x80000000u : 0xFFFFFFFFu));
}

template <int T>
struct LogprobLds {
    RowSums parts[T / kWave];
    float columns[T];
    uint32_t bests[64];
    float bound;
    int32_t groups[kLogprobGroupList];
    alignas(16) uint64_t cands[kLogprobCandidates];   // order of the logit, then the index backwards; zeros behind the last
    double log_s;
    float m;
    int32_t n_groups, n_cands;
    int32_t reached[32], equal[2][kWave];
    float best_x[T];
    int32_t best_i[T];
};

__device__ __forceinline__ float log_p(float x, float m, double log_s)
{
    return x == -__builtin_inff() ? x : (float)(((double)x - (double)m) - log_s);
}

// A row's outputs but the alternatives, by a wave that has its sums; returns log S.
__device__ __forceinline__ double finish_sums(const LogprobArgs& g, int64_t m, const RowSums& r, const Asked& a)
{
    const float inf = __builtin_inff();
    const bool empty = r.m == -inf;
    const double others = empty ? 0.0 : r.s + (double)(r.top - 1), log_s = log1p(others);
    if ((threadIdx.x & 63) == 0) {
        if (g.logprob != nullptr) g.logprob[m] = a.token < 0 ? 0.0f : a.inside ? log_p(a.mine, r.m, log_s) : -inf;
        if (g.rank != nullptr) g.rank[m] = a.token < 0 ? -1 : a.inside ? r.ahead : g.V;
        if (g.entropy != nullptr) g.entropy[m] = empty ? 0.0f : (float)(log_s - r.t / (1.0 + others));
    }
    return log_s;
}

// The K-th largest order of 64, without its 6 lowest bits, where the lane's
// number makes all different: a bound from below of the K-th largest logit, if
// the 64 are maxima of disjoint sets.
__device__ __forceinline__ uint32_t lane_order(float x) { return (float_order(x) & ~63u) | (threadIdx.x & 63); }

__device__ __forceinline__ float kth_bound(uint32_t mine, const uint32_t (&all)[64], int K)
{
    int place = 0;
#pragma unroll 16
    for (int j = 0; j < 64; ++j) place += all[j] > mine ? 1 : 0;
    const int lane = (int)__builtin_ctzll(__ballot(place == K - 1));
    const uint32_t order = (uint32_t)__builtin_amdgcn_readlane((int)mine, lane) & ~63u;
    return order > 0x007FFFFFu ? order_float(order) : -__builtin_inff();   // (-inf's order; none below it is a number's)
}

// How many of the n keys are larger; the list ends in zeros up to a multiple of 16.
__device__ __forceinline__ int key_place(const uint64_t* keys, int n, uint64_t own)
{
    int place = 0;
    for (int j = 0; j < n; j += 16)
#pragma unroll
        for (int k = 0; k < 16; ++k) place += keys[j + k] > own ? 1 : 0;
    return place;
}

// A row's outputs, by a workgroup of T threads: sum_of() gives a wave the row's
// sums (behind the first barrier), largest[] are a thread's groups' maxima,
// number i * T + thread of those that the walk's TW threads wrote, of which there
// are `rows` times T at most.
template <bool F32, int T, int TW, int NG, typename SumOf>
__device__ __forceinline__ void finish_row(const LogprobArgs& g, int64_t m, const Asked& a, const float (&largest)[NG],
                                           int rows, LogprobLds<T>& lds, SumOf sum_of)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float inf = __builtin_inff();
    const uint8_t* row = row_of<F32>(g, m);
    const int K = g.topk;
    if (K == 0) {
        __syncthreads();
        if (wave == T / kWave - 1) finish_sums(g, m, sum_of(), a);
        return;
    }
    float best = -inf;
#pragma unroll
    for (int c = 0; c < NG; c += 8)
        if (c < rows)
#pragma unroll
            for (int i = c; i < c + 8; ++i) best = fmaxf(best, largest[i]);
    lds.columns[tid] = best;
    if (tid == 0) lds.n_groups = lds.n_cands = 0;
    for (int c = tid; c < kLogprobCandidates; c += T) lds.cands[c] = 0;
    __syncthreads();
    if (wave == 0) {                                     // (one wave: they would all be at the same work, in turn)
        float column = lds.columns[lane];
#pragma unroll
        for (int i = 1; i < T / 64; ++i) column = fmaxf(column, lds.columns[lane + 64 * i]);
        const uint32_t order = lane_order(column);
        lds.bests[lane] = order;
        __builtin_amdgcn_wave_barrier();
        const float bound = kth_bound(order, lds.bests, K);
        if (lane == 0) lds.bound = bound > -inf ? bound : -kLargestLogit;   // (-inf itself is not available)
    }
    __syncthreads();
    const float bound = lds.bound;
    if (best >= bound) {
#pragma unroll
        for (int c = 0; c < NG; c += 8)
            if (c < rows) {
                uint32_t hits = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) hits |= largest[c + i] >= bound ? 1u << i : 0u;
                while (hits != 0) {
                    const int i = __builtin_ctz(hits);
                    hits &= hits - 1;
                    const int at = atomicAdd(&lds.n_groups, 1);
                    if (at < kLogprobGroupList) lds.groups[at] = (c + i) * T + tid;
                }
            }
    }
    __syncthreads();
    const int n_groups = lds.n_groups;
    if (wave == T / kWave - 1) {                         // the sums, while the other waves read the groups again
        const RowSums r = sum_of();
        const double log_s = finish_sums(g, m, r, a);
        if (lane == 0) {
            lds.m = r.m;
            lds.log_s = log_s;
        }
    } else if (n_groups <= kLogprobGroupList) {
        for (int j = tid; j < n_groups * 16; j += T - kWave) {
            const int group = lds.groups[j >> 4], in = j & 15;
            const int64_t first = (int64_t)(group / TW) * g.group_segments * (16 * TW) + (group % TW >> 6) * 1024 +
                                  logit_place<F32>(group & 63, in);
            for (int q = 0; q < g.group_segments; ++q) {
                const int64_t p = first + q * (16 * TW);
                if (p >= g.V) break;
                const float x = logit_at(row, F32, (size_t)p);
                if (x >= bound) {
                    const int at = atomicAdd(&lds.n_cands, 1);
                    if (at < kLogprobCandidates) lds.cands[at] = (uint64_t)float_order(x) << 32 | (uint32_t)~p;
                }
            }
        }
    }
    __syncthreads();
    const float row_m = lds.m;
    const double log_s = lds.log_s;
    auto put = [&](int k, float x, int i) {
        g.topk_ids[m * K + k] = i;
        g.topk_logprob[m * K + k] = i < 0 ? -inf : log_p(x, row_m, log_s);
    };
    const int n_cands = lds.n_cands;
    if (n_groups <= kLogprobGroupList && n_cands <= kLogprobCandidates) {
        for (int c = tid; c < n_cands; c += T) {
            const uint64_t own = lds.cands[c];
            const int at = key_place(lds.cands, n_cands, own);
            if (at < K) put(at, order_float((uint32_t)(own >> 32)), (int)~(uint32_t)own);
        }
        for (int k = n_cands + tid; k < K; k += T) put(k, -inf, -1);
        return;
    }
    // Too many reach the bound, which is a value that many logits share (masks of a
    // finite value, flat rows).  The K-th largest of the groups' maxima itself, bit
    // by bit from the top (of the order of -inf there are always K):
    __syncthreads();
    int id = tid;                                        // (made opaque: what follows from it would be kept through all rows, spilled)
    asm volatile("" : "+v"(id));
    const int at_lane = id & 63;
    if (id < 32) lds.reached[id] = 0;
    if (id == 0) lds.n_groups = lds.n_cands = 0;
    for (int c = id; c < kLogprobCandidates; c += T) lds.cands[c] = 0;
    __syncthreads();
    uint32_t kth = 0;
    int at_least = 0;                                    // groups whose maximum is that or more
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t trial = kth | 1u << bit;
        int n = 0;
#pragma unroll
        for (int c = 0; c < NG; c += 8)
            if (c < rows)
#pragma unroll
                for (int i = c; i < c + 8; ++i) n += __popcll(__ballot(float_order(largest[i]) >= trial));
        if (at_lane == 0 && n > 0) atomicAdd(&lds.reached[bit], n);
        __syncthreads();
        if (lds.reached[bit] >= K) {
            kth = trial;
            at_least = lds.reached[bit];
        }
    }
    // Larger logits stand in groups of a larger maximum, of which there are fewer
    // than K; they come first.  Where the groups that reach it are few, too (it is
    // one of the logits that few are left of), those that equal it come with them.
    const int span = 16 * g.group_segments;
    const uint32_t above = (int64_t)at_least * span <= kLogprobCandidates ? kth - 1 : kth;
#pragma unroll
    for (int c = 0; c < NG; c += 8)
        if (c < rows)
#pragma unroll
            for (int i = c; i < c + 8; ++i)
                if (float_order(largest[i]) > above) lds.groups[atomicAdd(&lds.n_groups, 1)] = i * T + id;
    __syncthreads();
    const int n_read = lds.n_groups * span;
    auto each_larger = [&](auto f) {
        for (int j = id; j < n_read; j += T) {
            const int group = lds.groups[j / span], in = j % span;
            const int64_t p = ((int64_t)(group / TW) * g.group_segments + (in >> 4)) * (16 * TW) + (group % TW >> 6) * 1024 +
                              logit_place<F32>(group & 63, in & 15);
            if (p >= g.V) continue;
            const float x = logit_at(row, F32, (size_t)p);
            if (float_order(x) > above) f(x, (int)p);
        }
    };
    each_larger([&](float x, int p) {
        const int at = atomicAdd(&lds.n_cands, 1);
        if (at < kLogprobCandidates) lds.cands[at] = (uint64_t)float_order(x) << 32 | (uint32_t)~p;
    });
    __syncthreads();
    const int larger = lds.n_cands;
    if (larger <= kLogprobCandidates) {
        for (int c = id; c < larger; c += T) {
            const uint64_t own = lds.cands[c];
            const int at = key_place(lds.cands, larger, own);
            if (at < K) put(at, order_float((uint32_t)(own >> 32)), (int)~(uint32_t)own);
        }
    } else {
        // (groups of several segments that are large throughout) one after another:
        // the first of those behind the last one
        float x = inf;
        int i = -1;
        for (int k = 0; k < K; ++k) {
            float bx = -inf;
            int bi = -1;
            each_larger([&](float c, int v) {
                if (logit_before(x, i, c, v) && (bi < 0 || logit_before(c, v, bx, bi))) {
                    bx = c;
                    bi = v;
                }
            });
            __syncthreads();
            lds.best_x[id] = bx;
            lds.best_i[id] = bi;
            __syncthreads();
            for (int half = T / 2; half > 0; half >>= 1) {
                if (id < half) {
                    const float ox = lds.best_x[id + half];
                    const int oi = lds.best_i[id + half];
                    if (oi >= 0 && (lds.best_i[id] < 0 || logit_before(ox, oi, lds.best_x[id], lds.best_i[id]))) {
                        lds.best_x[id] = ox;
                        lds.best_i[id] = oi;
                    }
                }
                __syncthreads();
            }
            x = lds.best_x[0];
            i = lds.best_i[0];
            if (id == 0) put(k, x, i);
        }
        return;
    }
    // Then the first of those that equal it: 64 pieces of a wave's 64 logits at a
    // time, counted, until there are enough.
    constexpr int W = T / kWave, U = kWave / W;
    const float tie = order_float(kth);
    int found = larger;
    for (int64_t at = 0, turn = 0; tie > -inf && at < g.V && found < K; at += U * T, turn ^= 1) {
        uint64_t who[U];
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = logit_at(row, F32, (size_t)min(at + u * T + id, (int64_t)g.V - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            who[u] = __ballot(at + u * T + id < g.V && x[u] == tie);
            if (at_lane == 0) lds.equal[turn][u * W + wave] = __popcll(who[u]);
        }
        __syncthreads();
        const int mine = lds.equal[turn][at_lane];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (who[u] == 0) continue;
            const int to = found + wave_sum_i32(at_lane < u * W + wave ? mine : 0) +
                           (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who[u] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who[u], 0));
            if ((who[u] >> at_lane & 1) != 0 && to < K) put(to, tie, (int)(at + u * T + id));
        }
        found += wave_sum_i32(mine);
    }
    for (int k = found + id; k < K; k += T) put(k, -inf, -1);
}

// Walks the segments [s0, s1) of a row with the workgroup's T / 64 waves, 1,024
// logits each, and puts the groups' largest logits into `maxima`.  Returns the
// wave's sums.
template <bool F32, int T>
__device__ __forceinline__ RowSums walk_row(const LogprobArgs& g, int64_t m, int s0, int s1, float* maxima, Asked& a)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    LogitWalk<F32> w;
    w.row = row_of<F32>(g, m);
    w.V = g.V;
    w.lane = lane;
    Logits16<F32> now, next;
    auto at = [&](int s) { return s * (16 * T) + wave * 1024; };
    w.load(at(s0), now);
    a = asked_of<F32>(g, m, w.row);
    w.token = a.token;
    w.asked = g.rank != nullptr && a.inside;
    w.mine = a.mine;
    w.above = nextafterf(w.mine, __builtin_inff());
    float group = -__builtin_inff();
    int in = 0;
    for (int s = s0; s < s1; ++s) {
        if (s + 1 < s1) w.load(at(s + 1), next);
        group = fmaxf(group, w.add(at(s), now));
        if (++in == g.group_segments || s + 1 == s1) {
            if (g.topk > 0) maxima[(s / g.group_segments) * T + tid] = group;
            group = -__builtin_inff();
            in = 0;
        }
        now = next;
    }
    return w.sums();
}

__device__ __forceinline__ RowSums no_sums() { return RowSums{0.0, 0.0, -__builtin_inff(), 0, 0, 0}; }

// The largest logits of n groups, i * T + thread in largest[i].
template <int T, int NG>
__device__ __forceinline__ void load_maxima(const float* maxima, int n, float (&largest)[NG])
{
#pragma unroll
    for (int c = 0; c < NG; c += 8)
        if (c * T < n)
#pragma unroll
            for (int i = c; i < c + 8; ++i) largest[i] = maxima[min(i * T + (int)threadIdx.x, n - 1)];
#pragma unroll
    for (int i = 0; i < NG; ++i) largest[i] = i * T + (int)threadIdx.x < n ? largest[i] : -__builtin_inff();
}

// A workgroup of T threads a row, from the logits to the outputs: one launch and
// no workspace where there are rows enough (301 rows of 32,771 bf16: 15.7 us).
template <bool F32, int T>
__global__ __launch_bounds__(T, 4) void logprob_rows_kernel(LogprobArgs g)
{
    extern __shared__ float maxima[];                    // [groups][T]
    __shared__ LogprobLds<T> lds;
    const int lane = threadIdx.x & 63;
    for (int64_t m = blockIdx.x; m < g.M; m += gridDim.x) {
        Asked a;
        const RowSums r = walk_row<F32, T>(g, m, 0, g.segments, maxima, a);
        if (lane == 0) lds.parts[threadIdx.x >> 6] = r;
        float largest[16] = {};
        if (g.topk > 0) load_maxima<T>(maxima, g.groups * T, largest);   // (a thread reads what it wrote itself)
        finish_row<F32, T, T>(g, m, a, largest, g.groups, lds,
                              [&] { return join_sums(lane < T / kWave ? lds.parts[lane] : no_sums()); });
        __syncthreads();
    }
}

// A workgroup a part of a row: its sums and its groups' largest logits go to
// the workspace.  Fewer rows than 129 leave compute units idle otherwise: 64 of
// 157,184 bf16 as 13 parts each 17.6 us with the join, one of fp32 as 39 10.1 us
// (parts of 512 to 4,096 workgroups in all, and two segments ahead instead of
// one, made no difference).
template <bool F32>
__global__ __launch_bounds__(256, 5) void logprob_parts_kernel(LogprobArgs g)
{
    __shared__ RowSums parts[4];
    const int lane = threadIdx.x & 63;
    const int64_t m = blockIdx.x / g.parts;
    const int part = (int)(blockIdx.x - m * g.parts), s0 = part * g.part_segments;
    Asked a;
    const RowSums r = walk_row<F32, 256>(g, m, s0, min(s0 + g.part_segments, g.segments), g.maxima + m * g.groups * 256, a);
    if (lane == 0) parts[threadIdx.x >> 6] = r;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const RowSums all = join_sums(lane < 4 ? parts[lane] : no_sums());
    if (lane == 0) g.sums[m * g.parts + part] = all;
}

// A workgroup a row (a wave, where no alternatives are asked for), from its
// parts to the outputs.
template <bool F32>
__global__ __launch_bounds__(kLogprobJoin) void logprob_join_kernel(LogprobArgs g)
{
    constexpr int T = kLogprobJoin;
    __shared__ LogprobLds<T> lds;
    const int lane = threadIdx.x & 63, n = g.groups * 256;
    const int64_t m = blockIdx.x;
    float largest[kLogprobMaxParts * 256 / T] = {};
    if (g.topk > 0) load_maxima<T>(g.maxima + m * n, n, largest);
    const RowSums mine = lane < g.parts ? g.sums[m * g.parts + lane] : no_sums();
    const Asked a = asked_of<F32>(g, m, row_of<F32>(g, m));
    if (g.topk == 0) {
        finish_sums(g, m, join_sums(mine), a);
        return;
    }
    finish_row<F32, T, 256>(g, m, a, largest, (n + T - 1) / T, lds, [&] { return join_sums(mine); });
}

// A wave a row.  Where alternatives are asked for, a second wave finds them
// meanwhile, in two passes over the same row: one after the other they are two
// chains of thousands of cycles (12 rows of 192: 7.0 us, with two waves 4.1, of
// which the sums alone are 3.8; 4,096 of 1,000: 12 us).  ONE: a row of at most
// 1,024 logits; five workgroups a compute unit, as the rows with shared values
// would otherwise take registers for four and cost all others 5%.
template <bool F32, bool ONE>
__global__ __launch_bounds__(256, ONE ? 5 : 4) void logprob_short_kernel(LogprobArgs g)
{
    constexpr int E = Logits16<F32>::kVec;
    __shared__ uint32_t bests[2][64];
    __shared__ alignas(16) uint64_t cands[2][kLogprobShortList];
    __shared__ double log_sums[2];
    __shared__ float maxima[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), K = g.topk;
    const float inf = __builtin_inff();
    const int slot = K > 0 ? wave >> 1 : wave;
    const int64_t m = (int64_t)blockIdx.x * (K > 0 ? 2 : 4) + slot;
    const bool row = m < g.M, alternatives = K > 0 && (wave & 1) != 0;
    LogitWalk<F32> w;
    if (row) {
        w.row = row_of<F32>(g, m);
        w.V = g.V;
        w.lane = lane;
    }
    if (row && !alternatives) {
        Logits16<F32> now, next;
        w.load(0, now);
        const Asked a = asked_of<F32>(g, m, w.row);
        w.token = a.token;
        w.asked = g.rank != nullptr && a.inside;
        w.mine = a.mine;
        w.above = nextafterf(w.mine, inf);
        if constexpr (ONE) {
            w.add(0, now);
        } else {
#pragma unroll 1
            for (int at = 0; at < g.V; at += 1024) {
                if (at + 1024 < g.V) w.load(at + 1024, next);
                w.add(at, now);
                now = next;
            }
        }
        const RowSums r = w.sums();
        const double log_s = finish_sums(g, m, r, a);
        if (K > 0 && lane == 0) {
            log_sums[slot] = log_s;
            maxima[slot] = r.m;
        }
    }
    if (K == 0) return;
    Logits16<F32> raw, next;
    int n = 0, place[kLogprobShortList / 64];
    uint64_t own[kLogprobShortList / 64];
    auto key_of = [&](int at, int i) {                   // 0: no logit, or nothing above -inf
        const float x = logit_value(raw.get(i));
        const int p = at + logit_place<F32>(lane, i);
        return p < g.V && x > -inf ? (uint64_t)float_order(x) << 32 | (uint32_t)~p : 0ull;
    };
    // f of 1,024 logits at a time
    auto each = [&](auto f) {
        if constexpr (ONE) {
            f(0);
        } else {
            w.load(0, raw);
#pragma unroll 1
            for (int at = 0; at < g.V; at += 1024) {
                if (at + 1024 < g.V) w.load(at + 1024, next);
                f(at);
                raw = next;
            }
        }
    };
    float best = -inf;
    if (row && alternatives) {
        if constexpr (ONE) w.load(0, raw);
        each([&](int) {
#pragma unroll
            for (int i = 0; i < 16; ++i) best = fmaxf(best, logit_value(raw.get(i)));   // (behind the row: -inf)
        });
        bests[slot][lane] = lane_order(best);
#pragma unroll
        for (int c = 0; c < kLogprobShortList; c += 64) cands[slot][c + lane] = 0;
        __builtin_amdgcn_wave_barrier();
        const float bound = kth_bound(bests[slot][lane], bests[slot], K);
        const uint64_t least = bound > -inf ? (uint64_t)float_order(bound) << 32 : 1;
        each([&](int at) {
#pragma unroll
            for (int u = 0; u < 16; u += E) {
                if (at + u * 64 >= g.V) break;                // (u of 16 values of a lane: 64 u of the wave's)
#pragma unroll
                for (int i = u; i < u + E; ++i) {
                    const uint64_t key = key_of(at, i);
                    const uint64_t who = __ballot(key >= least);
                    if (who == 0) continue;
                    const int to = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
                    if (key >= least && to < kLogprobShortList) cands[slot][to] = key;
                    n += __popcll(who);
                }
            }
        });
        __builtin_amdgcn_wave_barrier();
        if (n <= kLogprobShortList)
#pragma unroll
            for (int c = 0; c < kLogprobShortList / 64; ++c) {
                own[c] = cands[slot][c * 64 + lane];
                place[c] = c * 64 < n ? key_place(cands[slot], n, own[c]) : K;
            }
    }
    __syncthreads();
    if (!row || !alternatives) return;
    const double log_s = log_sums[slot];
    const float row_m = maxima[slot];
    auto put = [&](int k, uint64_t key) {
        const bool none = key == 0;
        g.topk_ids[m * K + k] = none ? -1 : (int)~(uint32_t)key;
        g.topk_logprob[m * K + k] = none ? -inf : log_p(order_float((uint32_t)(key >> 32)), row_m, log_s);
    };
    if (n <= kLogprobShortList) {
#pragma unroll
        for (int c = 0; c < kLogprobShortList / 64; ++c)
            if (c * 64 + lane < n && place[c] < K) put(place[c], own[c]);
        for (int k = n + lane; k < K; k += 64) put(k, 0);
        return;
    }
    // Many share the bound's value: as in finish_row, with lanes for groups (1,024
    // rows of 6,000, all but a few at a finite value, 20 alternatives: 31 us, where
    // a pass for each took 152).
    bests[slot][lane] = float_order(best);
    __builtin_amdgcn_wave_barrier();
    int before = 0;
#pragma unroll 16
    for (int l = 0; l < 64; ++l) {
        const uint32_t other = bests[slot][l], mine = float_order(best);
        before += other > mine || (other == mine && l < lane) ? 1 : 0;
    }
    const uint32_t kth = (uint32_t)__builtin_amdgcn_readlane((int)float_order(best), (int)__builtin_ctzll(__ballot(before == K - 1)));
#pragma unroll
    for (int c = 0; c < kLogprobShortList; c += 64) cands[slot][c + lane] = 0;
    __builtin_amdgcn_wave_barrier();
    int larger = 0;
    each([&](int at) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint64_t key = key_of(at, i), who = __ballot((uint32_t)(key >> 32) > kth);
            if (who == 0) continue;
            const int to = larger + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
            if ((uint32_t)(key >> 32) > kth && to < kLogprobShortList) cands[slot][to] = key;
            larger += __popcll(who);
        }
    });
    __builtin_amdgcn_wave_barrier();
    if (larger > kLogprobShortList) {
        // (less than K lanes, but large throughout) the largest key below the last, K times
        uint64_t last = ~0ull;
        for (int k = 0; k < K; ++k) {
            uint64_t top = 0;
            each([&](int at) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t key = key_of(at, i);
                    if (key < last) top = max_u64(top, key);
                }
            });
            last = wave_max_u64(top);
            if (lane == 0) put(k, last);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < kLogprobShortList; c += 64) {
        const uint64_t key = cands[slot][c + lane];
        const int to = c < larger ? key_place(cands[slot], larger, key) : K;
        if (c + lane < larger && to < K) put(to, key);
    }
    int found = larger;
    each([&](int at) {
#pragma unroll
        for (int u = 0; u < 16; u += E) {
            if (found >= K) return;
            int ahead = 0, all = 0;                      // that stand before the lane's own, and in all
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint64_t who = __ballot((uint32_t)(key_of(at, u + e) >> 32) == kth);
                ahead += (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
                all += __popcll(who);
            }
            if (all == 0) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint64_t key = key_of(at, u + e);
                if ((uint32_t)(key >> 32) != kth) continue;
                if (found + ahead < K) put(found + ahead, key);
                ++ahead;
            }
            found += all;
        }
    });
    for (int k = found + lane; k < K; k += 64) put(k, 0);
}

}  // namespace moe
