// lora_kernels.hpp -- the adapters' two products: u of each token, and B u added
// to a projection's output (gfx950; lora_common.hpp says how tokens are taken).
#pragma once

#include "lora_common.hpp"

namespace moe {

// ---------------------------------------------------------------------------
// u of 16 tokens and 16 rows of A: 8 waves share K, their sums meet in LDS.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(512) void lora_shrink_kernel(LoraArgs g)
{
    constexpr int W = 8, U = 5;                          // waves; steps of 32 whose loads go out together
    __shared__ f32x4 part[W][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, k0 = (lane >> 4) * 8;
    const int ranks = g.rp / 16, slot = (int)(blockIdx.x % g.slots);
    const int64_t rest = blockIdx.x / g.slots, m0 = rest / ranks * 16;
    const int r0 = (int)(rest % ranks) * 16;
    const int id = adapter_of(g, m0 + row);
    const uint16_t* x = g.x + (size_t)min(m0 + row, g.M - 1) * g.K;
    const int whole = g.K / 32, s0 = whole * wave / W, s1 = whole * (wave + 1) / W;
    each_adapter(id, slot, g.slots, [&](int i, bool mine) {
        if (i < 0) return;
        const uint16_t* a = g.a + ((size_t)i * g.r + min(r0 + row, g.r - 1)) * g.K;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = s0; s < s1; s += U) {
            u32x4 av[U], xv[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int k = min(s + j, s1 - 1) * 32 + k0;
                av[j] = *reinterpret_cast<const u32x4_half*>(a + k);
                xv[j] = *reinterpret_cast<const u32x4_half*>(x + k);
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s + j < s1) acc = mfma(av[j], xv[j], acc);
        }
        if (whole * 32 < g.K && wave == W - 1)
            acc = mfma(load_bf16x8<false>(a, whole * 32 + k0, g.K), load_bf16x8<false>(x, whole * 32 + k0, g.K), acc);
        part[wave][lane] = acc;
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < W; ++w) acc += part[w][lane];
            const float scale = g.scale != nullptr ? g.scale[i] : 1.0f;
            const int rank = r0 + (lane >> 4) * 4;
            if (mine)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    g.u[(size_t)(m0 + row) * g.rp + rank + e] = rank + e < g.r ? acc[e] * scale : 0.0f;
        }
        __syncthreads();
    });
}

// 16 consecutive values of a row, n of them the row's, to and from fp32.
template <bool F32>
__device__ __forceinline__ void load_row16(const void* p, size_t at, int n, float (&v)[16])
{
    if (n >= 16) {
        if constexpr (F32) {
            const f32x4_word* q = reinterpret_cast<const f32x4_word*>(static_cast<const float*>(p) + at);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = q[i >> 2][i & 3];
        } else {
            const u32x4_half* q = reinterpret_cast<const u32x4_half*>(static_cast<const uint16_t*>(p) + at);
            const u32x4 d[2] = {q[0], q[1]};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t w = d[i >> 3][(i & 7) >> 1];
                v[i] = __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? load_typed(p, F32 ? kTypeF32 : kTypeBf16, at + i) : 0.0f;
    }
}

template <bool F32>
__device__ __forceinline__ void store_row16(void* p, size_t at, int n, const float (&v)[16])
{
    if (n >= 16) {
        if constexpr (F32) {
            f32x4_word* q = reinterpret_cast<f32x4_word*>(static_cast<float*>(p) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        } else {
            u32x4_half* q = reinterpret_cast<u32x4_half*>(static_cast<uint16_t*>(p) + at);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 d;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d[i] = f32_to_bf16_bits(v[8 * h + 2 * i]) | f32_to_bf16_bits(v[8 * h + 2 * i + 1]) << 16;
                q[h] = d;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (i < n) {
                if constexpr (F32) static_cast<float*>(p)[at + i] = v[i];
                else static_cast<uint16_t*>(p)[at + i] = (uint16_t)f32_to_bf16_bits(v[i]);
            }
    }
}

// ---------------------------------------------------------------------------
// out of TM x 16 tokens and 256 channels, 64 a wave.  The channels are the
// first operand, row q of tile j being channel 16 (q / 4) + 4 j + q % 4, so that
// a lane gets 16 consecutive channels of its token over the four tiles.  B's
// rows stay in registers while the adapter is the same.  RK: steps of 32 ranks.
// ---------------------------------------------------------------------------
template <bool F32, int RK, bool EVEN>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs g)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, k0 = (lane >> 4) * 8;
    const int64_t tiles = (g.N + 255) / 256;
    const int slot = (int)(blockIdx.x % g.slots);
    const int64_t rest = blockIdx.x / g.slots, m_tile = rest / tiles * g.token_tiles * 16;
    const int64_t n0 = (rest % tiles) * 256 + wave * 64, n = n0 + (lane >> 4) * 16;
    if (n0 >= g.N) return;
    const int left = (int)min((int64_t)16, g.N - n);     // channels of this lane (may be none)
    u32x4 bv[4][RK];
    int held = -1;
    for (int t = 0; t < g.token_tiles; ++t) {
        const int64_t m = m_tile + t * 16 + row;
        if (m_tile + t * 16 >= g.M) return;
        const int id = adapter_of(g, m);
        const size_t at = (size_t)min(m, g.M - 1) * g.N + min(n, g.N - 1);
        float o[16] = {};
        if (g.base != nullptr) load_row16<F32>(g.base, at, left, o);
        bool own = false;
        each_adapter(id, slot, g.slots, [&](int i, bool mine) {
            own |= mine;
            if (i < 0) return;
            if (i != held) {
                held = i;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t c = min(n0 + (row >> 2) * 16 + j * 4 + (row & 3), g.N - 1);
                    const uint16_t* b = g.b + ((size_t)i * g.N + c) * g.r;
#pragma unroll
                    for (int k = 0; k < RK; ++k) bv[j][k] = load_bf16x8<EVEN>(b, 32 * k + k0, g.r);
                }
            }
            f32x4 acc[4] = {};
            const float* u = g.u + (size_t)min(m, g.M - 1) * g.rp + k0;
#pragma unroll
            for (int k = 0; k < RK; ++k) {
                if (k * 32 >= g.rp) break;
                // (a token of another adapter has its own u here, and drops the result)
                const Split3 s = split_u(u + 32 * k);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int p = 2; p >= 0; --p) acc[j] = mfma(bv[j][k], s.v[p], acc[j]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] += mine ? acc[e >> 2][e & 3] : 0.0f;
        });
        if (own && left > 0) store_row16<F32>(g.out, at, left, o);
    }
}

}  // namespace moe
