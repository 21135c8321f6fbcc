// logprob_kernels.hpp -- log probabilities of given tokens, with rank, entropy
// and top alternatives (gfx950).
//
// Of a row of logits l (NaN as -inf, +inf as the largest finite fp32), with
// m = max l, S = sum exp(l - m) and T = sum exp(l - m) (l - m):
//   log p(v) = (l_v - m) - log S,   entropy = -sum p log p = log S - T / S,
//   rank(t)  = how many v have l_v > l_t, or l_v = l_t and v < t.
// The largest logit's own 1 is kept out of S's sum: in a confident row log S =
// log1p(S - 1) is what the others are beside it, which fp32 would lose.
#pragma once

#include "around_common.hpp"

namespace moe {

// A logit's value as the definitions count it.
__device__ __forceinline__ float logit_value(float x)
{
    return x != x ? -__builtin_inff() : __builtin_fminf(x, 3.40282347e38f) + 0.0f;   // (+ 0: no -0)
}

// Whether (x, i) stands before (y, j): larger, or equal with a lower index.
__device__ __forceinline__ bool logit_before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

// One workgroup a row; each thread strides over it, once for the maximum, once
// for the sums and the rank, and once for each alternative.
__global__ __launch_bounds__(256) void logprob_row_kernel(LogprobArgs g)
{
    __shared__ float part_x[4];
    __shared__ int part_i[4];
    __shared__ double part_s[4], part_t[4];
    const int tid = threadIdx.x, wave = tid >> 6;
    const float inf = __builtin_inff();
    for (int64_t m = blockIdx.x; m < g.M; m += gridDim.x) {
        const size_t row = (size_t)m * (size_t)g.stride;
        auto value = [&](int v) { return logit_value(load_typed(g.logits, g.type, row + v)); };
        // the first available of those behind (px, pi)
        auto next = [&](float px, int pi, float& x, int& i) {
            x = -inf;
            i = -1;
            for (int v = tid; v < g.V; v += 256) {
                const float c = value(v);
                if (c > -inf && logit_before(px, pi, c, v) && (i < 0 || logit_before(c, v, x, i))) {
                    x = c;
                    i = v;
                }
            }
            for (int o = 32; o > 0; o >>= 1) {
                const float ox = __shfl_xor(x, o);
                const int oi = __shfl_xor(i, o);
                if (oi >= 0 && (i < 0 || logit_before(ox, oi, x, i))) {
                    x = ox;
                    i = oi;
                }
            }
            __syncthreads();
            if ((tid & 63) == 0) {
                part_x[wave] = x;
                part_i[wave] = i;
            }
            __syncthreads();
            for (int w = 0; w < 4; ++w)
                if (part_i[w] >= 0 && (i < 0 || logit_before(part_x[w], part_i[w], x, i))) {
                    x = part_x[w];
                    i = part_i[w];
                }
        };
        float top;
        int at;
        next(inf, -1, top, at);
        const int token = g.tokens != nullptr ? g.tokens[m] : -1;
        const bool asked = token >= 0 && token < g.V;
        const float mine = asked ? value(token) : 0.0f;
        double s = 0.0, t = 0.0;                         // without the largest
        int rank = 0;
        for (int v = tid; v < g.V; v += 256) {
            const float c = value(v);
            if (asked && logit_before(c, v, mine, token)) ++rank;
            if (at < 0 || v == at || c == -inf) continue;
            const double d = (double)c - (double)top, e = exp(d);
            s += e;
            if (e > 0.0) t += e * d;
        }
        s = wave_sum_f64(s);
        t = wave_sum_f64(t);
        for (int o = 32; o > 0; o >>= 1) rank += __shfl_xor(rank, o);
        __syncthreads();
        if ((tid & 63) == 0) {
            part_s[wave] = s;
            part_t[wave] = t;
            part_i[wave] = rank;
        }
        __syncthreads();
        s = (part_s[0] + part_s[1]) + (part_s[2] + part_s[3]);
        t = (part_t[0] + part_t[1]) + (part_t[2] + part_t[3]);
        rank = part_i[0] + part_i[1] + part_i[2] + part_i[3];
        const double log_s = log1p(s);
        auto log_p = [&](float x) { return x == -inf ? -inf : (float)(((double)x - (double)top) - log_s); };
        if (tid == 0) {
            if (g.logprob != nullptr) g.logprob[m] = token < 0 ? 0.0f : asked ? log_p(mine) : -inf;
            if (g.rank != nullptr) g.rank[m] = token < 0 ? -1 : asked ? rank : g.V;
            if (g.entropy != nullptr) g.entropy[m] = at < 0 ? 0.0f : (float)(log_s - t / (1.0 + s));
        }
        float x = inf;
        int i = -1;
        for (int k = 0; k < g.topk; ++k) {
            float nx = -inf;
            int ni = -1;
            if (k == 0 || i >= 0) next(x, i, nx, ni);
            x = nx;
            i = ni;
            if (tid == 0) {
                g.topk_ids[m * g.topk + k] = i;
                g.topk_logprob[m * g.topk + k] = i < 0 ? -inf : log_p(x);
            }
        }
        __syncthreads();
    }
}

}  // namespace moe
