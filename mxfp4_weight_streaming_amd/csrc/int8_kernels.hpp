// int8_kernels.hpp -- the int8 matrix product (gfx950):
//   out[m,n] = (sum_k a[m,k] w[n,k]) * a_scale[m] * w_scale[n]
// summed exactly in int32, so no order of the sum changes the result.
#pragma once

#include "around_common.hpp"

namespace moe {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// 16 codes of row r at column k, 0 outside the matrix.  Rows of a K that is no
// multiple of 16 start at any address, so those load byte by byte.
__device__ __forceinline__ u32x4 int8_load16(const uint8_t* p, int64_t r, int64_t rows, int k, int K)
{
    if (r >= rows || k >= K) return u32x4{0, 0, 0, 0};
    const uint8_t* src = p + (size_t)r * K + k;
    if (K % 16 == 0) return *reinterpret_cast<const u32x4*>(src);
    uint32_t d[4] = {0, 0, 0, 0};
    const int n = min(16, K - k);
    for (int i = 0; i < n; ++i) d[i >> 2] |= (uint32_t)src[i] << (8 * (i & 3));
    return u32x4{d[0], d[1], d[2], d[3]};
}

__device__ __forceinline__ void int8_store(const Int8Args& g, int64_t m, int64_t n, int32_t acc)
{
    if (m >= g.M || n >= g.N) return;
    const float v = ((float)acc * g.a_scale[m]) * g.w_scale[n];
    const size_t at = (size_t)m * g.N + n;
    if (g.out_type == kTypeF32) static_cast<float*>(g.out)[at] = v;
    else static_cast<uint16_t*>(g.out)[at] = (uint16_t)f32_to_bf16_bits(v);
}

// 64 x 64 output tile a workgroup, 32 x 32 a wave, 64 columns of K a step.
constexpr int kInt8Tile = 64;

__global__ __launch_bounds__(256) void int8_linear_kernel(Int8Args g)
{
    __shared__ u32x4 al[kInt8Tile][5], wl[kInt8Tile][5];   // 64 codes a row, padded by 16 bytes
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    const int64_t nt = (g.N + kInt8Tile - 1) / kInt8Tile, tiles = nt * ((g.M + kInt8Tile - 1) / kInt8Tile);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m0 = t / nt * kInt8Tile, n0 = t % nt * kInt8Tile;
        i32x4 acc[2][2] = {};
        for (int k0 = 0; k0 < g.K; k0 += 64) {
            __syncthreads();
            al[tid >> 2][tid & 3] = int8_load16(g.a, m0 + (tid >> 2), g.M, k0 + (tid & 3) * 16, g.K);
            wl[tid >> 2][tid & 3] = int8_load16(g.w, n0 + (tid >> 2), g.N, k0 + (tid & 3) * 16, g.K);
            __syncthreads();
            // lane l: row l % 16, codes 16 (l / 16) ... of the step, of both operands
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        __builtin_bit_cast(i32x4, al[wm + i * 16 + (lane & 15)][lane >> 4]),
                        __builtin_bit_cast(i32x4, wl[wn + j * 16 + (lane & 15)][lane >> 4]), acc[i][j], 0, 0, 0);
        }
        // lane l, register r: row 4 (l / 16) + r of a, row l % 16 of w
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    int8_store(g, m0 + wm + i * 16 + (lane >> 4) * 4 + r, n0 + wn + j * 16 + (lane & 15), acc[i][j][r]);
    }
}

}  // namespace moe
