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
// is ranked by counting.  Rows where more than a list's worth reach the bound
// (equal logits) take their alternatives one after another.
#pragma once

#include <type_traits>

#include "around_common.hpp"

namespace moe {

constexpr int kLogprobGroupList = 256;      // groups read again
constexpr int kLogprobCandidates = 512;     // logits ranked

// A logit's value as the definitions count it.
__device__ __forceinline__ float logit_value(float x)
{
    return x != x ? -__builtin_inff() : __builtin_fminf(x, 3.40282347e38f) + 0.0f;   // (+ 0: no -0)
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
    __device__ __forceinline__ void set(int i, float x)
    {
        if constexpr (F32) v[i >> 2][i & 3] = __float_as_uint(x);
        else if (i & 1) v[i >> 3][(i & 7) >> 1] |= __float_as_uint(x) & 0xFFFF0000u;
        else v[i >> 3][(i & 7) >> 1] = __float_as_uint(x) >> 16;
    }
};

typedef uint32_t u32x4_at __attribute__((ext_vector_type(4), aligned(2)));   // at any element

// Element i (0..15) of lane `lane`, in the wave's 1,024.
template <bool F32>
__device__ __forceinline__ int logit_place(int lane, int i)
{
    constexpr int E = Logits16<F32>::kVec;
    return (i / E) * (64 * E) + lane * E + i % E;
}

// A wave's walk over its segments of one row's part.
template <bool F32>
struct LogitWalk {
    const uint8_t* row;
    int V, lane;
    // given token
    int token;
    bool asked;
    float mine, above;                                   // its logit, and the next larger number
    // state: s and t a lane, the rest the wave's
    double s = 0.0, t = 0.0;
    float m = -__builtin_inff();
    int top = 0, ahead = 0;

    __device__ __forceinline__ void load(int at, Logits16<F32>& x) const
    {
        constexpr int E = Logits16<F32>::kVec, B = F32 ? 4 : 2;
        if (at + 1024 <= V) {
#pragma unroll
            for (int u = 0; u < Logits16<F32>::kVecs; ++u)
                x.v[u] = *reinterpret_cast<const u32x4_at*>(row + (size_t)(at + (u * 64 + lane) * E) * B);
            return;
        }
#pragma unroll
        for (int u = 0; u < Logits16<F32>::kVecs; ++u) {
            const int p = at + (u * 64 + lane) * E;
            if (p + E <= V) {
                x.v[u] = *reinterpret_cast<const u32x4_at*>(row + (size_t)p * B);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x.set(u * E + e, p + e < V ? load_typed(row, F32 ? kTypeF32 : kTypeBf16, p + e) : -__builtin_inff());
            }
        }
    }

    // Adds the 1,024 logits from `at`; returns the lane's largest.
    __device__ __forceinline__ float add(int at, const Logits16<F32>& raw)
    {
        const float inf = __builtin_inff();
        float x[16];
        float largest = -inf;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = logit_value(raw.get(i));
            largest = fmaxf(largest, x[i]);
        }
        if (asked) {
            if (at + 1024 <= V && (token >= at + 1024 || token < at)) {
                // before the token equal logits count, behind it only larger ones
                const float bar = token < at ? above : mine;
                int below = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) below += __popcll(__ballot(x[i] < bar));
                ahead += 1024 - below;
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int p = at + logit_place<F32>(lane, i);
                    ahead += __popcll(__ballot(p < V && logit_before(x[i], p, mine, token)));
                }
            }
        }
        bool equal = false;                              // whether a logit may equal m
        if (__any(largest >= m)) {
            const float most = wave_max(largest);
            if (most > m) {
                if (m > -inf) {
                    if (lane == 0) s += (double)top;
                    const double d = (double)m - (double)most, f = exp(d);
                    t = (t + s * d) * f;
                    s *= f;
                }
                m = most;
                top = 0;
            }
            if (m == -inf) return largest;               // nothing yet
            equal = true;
        }
        float ss[4] = {0.0f, 0.0f, 0.0f, 0.0f}, tt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        auto sums = [&](auto exclude) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // (-256: e^y is 0 there and far above, and stays so for -inf)
                const float y = fmaxf(x[i] - m, -256.0f);
                float e = __builtin_amdgcn_exp2f(y * 1.44269504f);
                if (exclude) {
                    top += __popcll(__ballot(x[i] == m));
                    e = x[i] == m ? 0.0f : e;
                }
                ss[i & 3] += e;
                tt[i & 3] = fmaf(e, y, tt[i & 3]);
            }
        };
        if (equal) sums(std::true_type{});
        else sums(std::false_type{});
        s += (double)((ss[0] + ss[1]) + (ss[2] + ss[3]));
        t += (double)((tt[0] + tt[1]) + (tt[2] + tt[3]));
        return largest;
    }

    __device__ __forceinline__ RowSums sums() const
    {
        return RowSums{wave_sum_f64(s), wave_sum_f64(t), m, top, ahead, 0};
    }
};

struct LogprobLds {
    RowSums parts[4];
    float columns[64 * 4];
    float bests[64];
    int32_t groups[kLogprobGroupList];
    float cand_x[kLogprobCandidates];
    int32_t cand_i[kLogprobCandidates];
    int32_t n_groups, n_cands;
};

// A row's outputs, by a workgroup of 256 threads: from its sums, the largest
// logit of each thread's groups (`best`) and of every group (`maxima`, group g
// of thread i at g * 256 + i).
template <bool F32>
__device__ __forceinline__ void finish_row(const LogprobArgs& g, int64_t m, const RowSums& r, float best,
                                           const float* maxima, LogprobLds& lds)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float inf = __builtin_inff();
    const uint8_t* row = static_cast<const uint8_t*>(g.logits) + (size_t)m * (size_t)g.stride * (F32 ? 4 : 2);
    const bool empty = r.m == -inf;
    const double others = empty ? 0.0 : r.s + (double)(r.top - 1), log_s = log1p(others);
    auto log_p = [&](float x) { return x == -inf ? -inf : (float)(((double)x - (double)r.m) - log_s); };
    if (tid == 0) {
        const int token = g.tokens != nullptr ? g.tokens[m] : -1;
        const bool asked = token >= 0 && token < g.V;
        if (g.logprob != nullptr) g.logprob[m] = token < 0 ? 0.0f : asked ? log_p(logit_at(row, F32, token)) : -inf;
        if (g.rank != nullptr) g.rank[m] = token < 0 ? -1 : asked ? r.ahead : g.V;
        if (g.entropy != nullptr) g.entropy[m] = empty ? 0.0f : (float)(log_s - r.t / (1.0 + others));
    }
    const int K = g.topk;
    if (K == 0) return;
    auto put = [&](int k, float x, int i) {
        g.topk_ids[m * K + k] = i;
        g.topk_logprob[m * K + k] = i < 0 ? -inf : log_p(x);
    };
    // the bound: the K-th largest of 64 columns' maxima
    lds.columns[tid] = best;
    if (tid == 0) lds.n_groups = lds.n_cands = 0;
    __syncthreads();
    const float column = fmaxf(fmaxf(lds.columns[lane], lds.columns[lane + 64]),
                               fmaxf(lds.columns[lane + 128], lds.columns[lane + 192]));
    if (wave == 0) lds.bests[lane] = column;
    __syncthreads();
    int place = 0;
#pragma unroll
    for (int j = 0; j < 64; ++j) place += logit_before(lds.bests[j], j, column, lane) ? 1 : 0;
    const float bound = row_lane(column, (int)__builtin_ctzll(__ballot(place == K - 1)));
    const int n = g.groups * 256;
    if (best >= bound && best > -inf)
        for (int i = tid; i < n; i += 256) {
            const float x = maxima[i];
            if (x >= bound && x > -inf) {
                const int at = atomicAdd(&lds.n_groups, 1);
                if (at < kLogprobGroupList) lds.groups[at] = i;
            }
        }
    __syncthreads();
    const int n_groups = lds.n_groups, each = 16 * g.group_segments;
    if (n_groups <= kLogprobGroupList) {
        for (int j = tid; j < n_groups * each; j += 256) {
            const int group = lds.groups[j / each], in = j % each;
            const int64_t p = ((int64_t)(group >> 8) * g.group_segments + (in >> 4)) * kLogprobSegment +
                              ((group & 255) >> 6) * 1024 + logit_place<F32>(group & 63, in & 15);
            if (p >= g.V) continue;
            const float x = logit_at(row, F32, (size_t)p);
            if (x >= bound && x > -inf) {
                const int at = atomicAdd(&lds.n_cands, 1);
                if (at < kLogprobCandidates) {
                    lds.cand_x[at] = x;
                    lds.cand_i[at] = (int)p;
                }
            }
        }
    }
    __syncthreads();
    const int n_cands = lds.n_cands;
    if (n_groups <= kLogprobGroupList && n_cands <= kLogprobCandidates) {
        for (int c = tid; c < n_cands; c += 256) {
            const float x = lds.cand_x[c];
            const int i = lds.cand_i[c];
            int at = 0;
            for (int j = 0; j < n_cands; ++j) at += logit_before(lds.cand_x[j], lds.cand_i[j], x, i) ? 1 : 0;
            if (at < K) put(at, x, i);
        }
        for (int k = n_cands + tid; k < K; k += 256) put(k, -inf, -1);
        return;
    }
    // one after another: the first of those behind the last one
    float x = inf;
    int i = -1;
    for (int k = 0; k < K; ++k) {
        float bx = -inf;
        int bi = -1;
        if (k == 0 || i >= 0) {
            for (int v = tid; v < g.V; v += 256) {
                const float c = logit_at(row, F32, (size_t)v);
                if (c > -inf && logit_before(x, i, c, v) && (bi < 0 || logit_before(c, v, bx, bi))) {
                    bx = c;
                    bi = v;
                }
            }
            __syncthreads();
            lds.cand_x[tid] = bx;
            lds.cand_i[tid] = bi;
            __syncthreads();
            for (int half = 128; half > 0; half >>= 1) {
                if (tid < half) {
                    const float ox = lds.cand_x[tid + half];
                    const int oi = lds.cand_i[tid + half];
                    if (oi >= 0 && (lds.cand_i[tid] < 0 || logit_before(ox, oi, lds.cand_x[tid], lds.cand_i[tid]))) {
                        lds.cand_x[tid] = ox;
                        lds.cand_i[tid] = oi;
                    }
                }
                __syncthreads();
            }
            bx = lds.cand_x[0];
            bi = lds.cand_i[0];
        }
        x = bx;
        i = bi;
        if (tid == 0) put(k, x, i);
    }
}

// Walks the segments [s0, s1) of a row with the workgroup's four waves, puts
// the groups' largest logits into `maxima`, and returns the thread's largest;
// the waves' sums go to LDS.
template <bool F32>
__device__ __forceinline__ float walk_row(const LogprobArgs& g, int64_t m, int s0, int s1, float* maxima, LogprobLds& lds)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    LogitWalk<F32> w;
    w.row = static_cast<const uint8_t*>(g.logits) + (size_t)m * (size_t)g.stride * (F32 ? 4 : 2);
    w.V = g.V;
    w.lane = lane;
    Logits16<F32> now, next;
    auto at = [&](int s) { return s * kLogprobSegment + wave * 1024; };
    w.load(at(s0), now);
    w.token = g.tokens != nullptr ? g.tokens[m] : -1;
    w.asked = g.rank != nullptr && w.token >= 0 && w.token < g.V;
    w.mine = w.asked ? logit_at(w.row, F32, w.token) : 0.0f;
    w.above = nextafterf(w.mine, __builtin_inff());
    float best = -__builtin_inff(), group = best;
    int in = 0;
    for (int s = s0; s < s1; ++s) {
        if (s + 1 < s1) w.load(at(s + 1), next);
        group = fmaxf(group, w.add(at(s), now));
        if (++in == g.group_segments || s + 1 == s1) {
            if (g.topk > 0) maxima[(s / g.group_segments) * 256 + tid] = group;
            best = fmaxf(best, group);
            group = -__builtin_inff();
            in = 0;
        }
        now = next;
    }
    const RowSums r = w.sums();
    if (lane == 0) lds.parts[wave] = r;
    return best;
}

__device__ __forceinline__ RowSums no_sums() { return RowSums{0.0, 0.0, -__builtin_inff(), 0, 0, 0}; }

// A workgroup a row, from the logits to the outputs.
template <bool F32>
__global__ __launch_bounds__(256) void logprob_rows_kernel(LogprobArgs g)
{
    extern __shared__ float maxima[];                    // [groups][256]
    __shared__ LogprobLds lds;
    const int lane = threadIdx.x & 63;
    for (int64_t m = blockIdx.x; m < g.M; m += gridDim.x) {
        const float best = walk_row<F32>(g, m, 0, g.segments, maxima, lds);
        __syncthreads();
        const RowSums r = join_sums(lane < 4 ? lds.parts[lane] : no_sums());
        finish_row<F32>(g, m, r, best, maxima, lds);
        __syncthreads();
    }
}

// A workgroup a part of a row: its sums and its groups' largest logits go to
// the workspace.
template <bool F32>
__global__ __launch_bounds__(256) void logprob_parts_kernel(LogprobArgs g)
{
    __shared__ LogprobLds lds;
    const int lane = threadIdx.x & 63;
    const int64_t m = blockIdx.x / g.parts;
    const int part = (int)(blockIdx.x - m * g.parts), s0 = part * g.part_segments;
    walk_row<F32>(g, m, s0, min(s0 + g.part_segments, g.segments), g.maxima + m * g.groups * 256, lds);
    __syncthreads();
    const RowSums r = join_sums(lane < 4 ? lds.parts[lane] : no_sums());
    if (threadIdx.x == 0) g.sums[m * g.parts + part] = r;
}

// A workgroup a row, from its parts to the outputs.
template <bool F32>
__global__ __launch_bounds__(256) void logprob_join_kernel(LogprobArgs g)
{
    __shared__ LogprobLds lds;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t m = blockIdx.x;
    const float* maxima = g.maxima + m * g.groups * 256;
    float best = -__builtin_inff();
    if (g.topk > 0)
        for (int i = tid; i < g.groups * 256; i += 256) best = fmaxf(best, maxima[i]);
    const RowSums r = join_sums(lane < g.parts ? g.sums[m * g.parts + lane] : no_sums());
    finish_row<F32>(g, m, r, best, maxima, lds);
}

}  // namespace moe
