// lora_kernels.hpp -- low-rank adapters of many requests (gfx950): token m has
// adapter i = ids[m], and
//   u[m] = scale[i] A[i] x[m]           (r values, fp32)
//   out[m] = round(base[m] + B[i] u[m])   base alone where i is no adapter
#pragma once

#include "around_common.hpp"

namespace moe {

// The adapter of token m, or -1.
__device__ __forceinline__ int adapter_of(const LoraArgs& g, int64_t m)
{
    const int i = g.ids[m];
    return i >= 0 && i < g.L ? i : -1;
}

// u: a wave a (token, row of A).
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs g)
{
    const int lane = threadIdx.x & 63;
    const int64_t rows = g.M * g.r;
    for (int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); p < rows; p += (int64_t)gridDim.x * 4) {
        const int64_t m = p / g.r;
        const int i = adapter_of(g, m);
        if (i < 0) continue;
        const uint16_t* x = g.x + (size_t)m * g.K;
        const uint16_t* a = g.a + ((size_t)i * g.r + (size_t)(p - m * g.r)) * g.K;
        float acc = 0.0f;
        for (int k = lane; k < g.K; k += 64) acc = fmaf(bf16_bits_to_f32(x[k]), bf16_bits_to_f32(a[k]), acc);
        acc = wave_sum(acc);
        if (lane == 0) g.u[p] = g.scale != nullptr ? acc * g.scale[i] : acc;
    }
}

// out: a thread an element.
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs g)
{
    const int64_t n_all = g.M * g.N;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < n_all; p += (int64_t)gridDim.x * 256) {
        const int64_t m = p / g.N, n = p - m * g.N;
        const int i = adapter_of(g, m);
        float v = g.base != nullptr ? load_typed(g.base, g.base_type, p) : 0.0f;
        if (i >= 0) {
            const uint16_t* b = g.b + ((size_t)i * g.N + n) * g.r;
            const float* u = g.u + m * g.r;
            float d = 0.0f;
            for (int j = 0; j < g.r; ++j) d = fmaf(u[j], bf16_bits_to_f32(b[j]), d);
            v += d;
        }
        if (g.out_type == kTypeF32) static_cast<float*>(g.out)[p] = v;
        else static_cast<uint16_t*>(g.out)[p] = (uint16_t)f32_to_bf16_bits(v);
    }
}

}  // namespace moe
