// norm_kernels.hpp -- residual add, RMS norm and 8-bit row quantisation in one
// kernel (gfx950).
//
//   r    = round_T(residual + x)          T: the residual's type
//   rstd = fl32(1 / sqrt(mean(r^2) + eps))   the sum of squares in fp64
//   y    = bf16(fl32(fl32(r w) rstd))
//   s    = amax|y| / 448 (E4M3) or / 127 (int8), 1 if 0;  q = code(y / s)
//
// The sum is kept in fp64 so that rstd is fl32 of the exact value whatever the
// order of the sum (but for one row in ~10^8): y, its codes and its scale then
// do not depend on how rows are split over lanes.
//
// amax needs no second pass: fl32(t rstd) and the rounding to bf16 do not
// decrease as t = |fl32(r w)| grows, so amax|y| = bf16(max t * rstd), and the
// sum and the maximum are reduced together.
#pragma once

#include "around_common.hpp"

namespace moe {

// Row scale of int8 codes, and the code of y / s: the quotient as in
// quant_div (product by the reciprocal, corrected once by its residual), whose
// rounding to a whole number equals the correctly rounded quotient's for every
// bf16 amax >= 2^-64 and bf16 |y| <= amax (checked on the host).
__device__ __forceinline__ QuantScale int8_scale(float amax)
{
    const float s = (amax == 0.0f) ? 1.0f : amax / 127.0f;
    return QuantScale{s, 1.0f / s, !(amax > 0.0f && amax < 0x1p-64f)};
}

__device__ __forceinline__ uint32_t int8_encode(float quotient)
{
    return (uint32_t)(int)__builtin_rintf(__builtin_amdgcn_fmed3f(quotient, -127.0f, 127.0f)) & 0xFFu;
}

// One row per workgroup pass, held in LDS as fp32; any H, any types.
constexpr int kNormThreads = 256;

__global__ __launch_bounds__(kNormThreads) void add_rmsnorm_kernel(NormArgs a)
{
#pragma clang fp contract(off)
    extern __shared__ float row[];                        // t = fl32(r w)
    __shared__ double part_ss[kNormThreads / kWave];
    __shared__ uint32_t part_max[kNormThreads / kWave];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t base = (size_t)m * a.H;
        double ss = 0.0;
        uint32_t top = 0;
        for (int i = tid; i < a.H; i += kNormThreads) {
            float r = load_typed(a.x, a.x_type, base + i);
            if (a.residual != nullptr) r = load_typed(a.residual, a.r_type, base + i) + r;
            if (a.r_type == kTypeBf16) r = round_to_bf16(r);
            if (a.residual_out != nullptr) {
                if (a.r_type == kTypeBf16) static_cast<uint16_t*>(a.residual_out)[base + i] = (uint16_t)f32_to_bf16_bits(r);
                else static_cast<float*>(a.residual_out)[base + i] = r;
            }
            ss += (double)r * (double)r;
            const float t = r * load_typed(a.weight, a.w_type, i);
            top = max(top, __float_as_uint(t) & 0x7FFFFFFFu);
            row[i] = t;
        }
        ss = wave_sum_f64(ss);
        top = wave_max_u32(top);
        if (lane == 0) {
            part_ss[wave] = ss;
            part_max[wave] = top;
        }
        __syncthreads();
        ss = (part_ss[0] + part_ss[1]) + (part_ss[2] + part_ss[3]);
        top = max(max(part_max[0], part_max[1]), max(part_max[2], part_max[3]));
        const float rstd = (float)(1.0 / sqrt(ss / (double)a.H + a.eps));
        const float amax = round_to_bf16(__uint_as_float(top) * rstd);
        const QuantScale qs = a.q_type == kQuantInt8 ? int8_scale(amax) : quant_scale(amax);
        for (int i = tid; i < a.H; i += kNormThreads) {
            const uint32_t yb = f32_to_bf16_bits(row[i] * rstd);
            if (a.y != nullptr) a.y[base + i] = (uint16_t)yb;
            if (a.q_type != kQuantNone) {
                const float v = quant_div(bf16_bits_to_f32(yb), qs);
                a.q[base + i] = (uint8_t)(a.q_type == kQuantInt8 ? int8_encode(v) : e4m3_encode(v));
            }
        }
        if (a.q_type != kQuantNone && tid == 0) a.scale[m] = qs.s;
        __syncthreads();                                  // the next row takes row[] and the parts
    }
}

// int8 codes and scales of the rows of a bf16 matrix: one wave a row.
__global__ __launch_bounds__(256) void int8_quantize_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                            uint8_t* __restrict__ q, float* __restrict__ scale)
{
    const int lane = threadIdx.x & 63;
    for (int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); m < rows; m += (int64_t)gridDim.x * 4) {
        const uint16_t* src = x + (size_t)m * cols;
        uint32_t top = 0;
        for (int i = lane; i < cols; i += kWave) top = max(top, (uint32_t)src[i] & 0x7FFFu);
        const QuantScale qs = int8_scale(bf16_bits_to_f32(wave_max_u32(top)));
        for (int i = lane; i < cols; i += kWave)
            q[(size_t)m * cols + i] = (uint8_t)int8_encode(quant_div(bf16_bits_to_f32(src[i]), qs));
        if (lane == 0) scale[m] = qs.s;
    }
}

}  // namespace moe
