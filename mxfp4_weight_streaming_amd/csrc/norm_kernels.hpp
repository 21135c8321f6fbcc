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

// Eight elements as they lie in memory, at any address: rows of an H that is no
// multiple of 8 start anywhere.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

template <bool F32>
struct Raw8 {
    u32x4 d[F32 ? 2 : 1];
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (F32) return __uint_as_float(d[j >> 2][j & 3]);
        const uint32_t v = d[0][j >> 1];
        return __uint_as_float(j & 1 ? v & 0xFFFF0000u : v << 16);
    }
    __device__ __forceinline__ void set(int j, float v)   // v already rounded to the type
    {
        if constexpr (F32) d[j >> 2][j & 3] = __float_as_uint(v);
        else if (j & 1) d[0][j >> 1] |= __float_as_uint(v) & 0xFFFF0000u;
        else d[0][j >> 1] = __float_as_uint(v) >> 16;
    }
};

// Elements i .. i + n - 1 (n = 8 but for a row's last, part vector).
template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* p, size_t i, int n)
{
    Raw8<F32> r;
    if (n == 8) {
        const u32x4_any* v = reinterpret_cast<const u32x4_any*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
        r.d[0] = v[0];
        if constexpr (F32) r.d[1] = v[1];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.set(j, j < n ? load_typed(p, F32 ? kTypeF32 : kTypeBf16, i + j) : 0.0f);
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, size_t i, int n, const Raw8<F32>& r)
{
    if (n == 8) {
        u32x4_any* v = reinterpret_cast<u32x4_any*>(static_cast<uint8_t*>(p) + i * (F32 ? 4 : 2));
        v[0] = r.d[0];
        if constexpr (F32) v[1] = r.d[1];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if constexpr (F32) static_cast<float*>(p)[i + j] = r.get(j);
                else static_cast<uint16_t*>(p)[i + j] = (uint16_t)(__float_as_uint(r.get(j)) >> 16);
            }
    }
}

// L threads a row (a DPP row of 16 lanes, a wave, or a workgroup of L), V
// vectors of 8 elements a thread: the whole row stays in registers between the
// reductions and the output, so each input is read once and nothing is read
// back.  (Beyond 16,384 elements, V = 8, not all of it: 34 registers a thread go
// to scratch memory where x and the residual are fp32, 2 where one of them is.)
template <int L>
struct RowParts {
    static constexpr int kWaves = L > kWave ? L / kWave : 1;
    double ss[kWaves];
    uint32_t top[kWaves];
};

// A row's sum of squares and largest magnitude, in every thread of the row.
template <int L>
__device__ __forceinline__ void reduce_row(double& ss, uint32_t& top, RowParts<L>& parts)
{
    if constexpr (L == 16) {
        ss = row_sum_f64(ss);
        top = row_max_u32(top);
    } else {
        ss = wave_sum_f64(ss);
        top = wave_max_u32(top);
    }
    if constexpr (L > kWave) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            parts.ss[wave] = ss;
            parts.top[wave] = top;
        }
        lds_barrier();
        ss = 0.0;
        top = 0;
#pragma unroll
        for (int k = 0; k < L / kWave; ++k) {
            ss += parts.ss[k];
            top = max(top, parts.top[k]);
        }
        lds_barrier();                                    // the next row takes the parts
    }
}

template <int L>
struct RowShape {
    static constexpr int kThreads = L < 256 ? 256 : L, kRows = kThreads / L;   // of a workgroup
};

__device__ __forceinline__ u32x2 encode8(const float* v, int q_type)
{
    if (q_type == kQuantE4m3) return u32x2{e4m3x4_encode(v[0], v[1], v[2], v[3]), e4m3x4_encode(v[4], v[5], v[6], v[7])};
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        c[h] = int8_encode(v[4 * h]) | int8_encode(v[4 * h + 1]) << 8 | int8_encode(v[4 * h + 2]) << 16 |
               int8_encode(v[4 * h + 3]) << 24;
    return c;
}

__device__ __forceinline__ void store_codes(uint8_t* q, size_t at, int n, u32x2 c)
{
    if (n == 8) *reinterpret_cast<u32x2_any*>(q + at) = c;
    else
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) q[at + j] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
}

// Bound by the rows' bytes once there are enough of them: 16,384 rows of 2,560
// (fp32 x, bf16 residual, y, E4M3 codes) 86-92 us, 5.0-5.3 TB/s, where a
// copy reaches 4.9 TB/s; one row 3.2 us in a graph, a launch and three memory
// latencies.  (The first kernel, a workgroup of 256 with the row in LDS and
// single elements a load, took 145 us.)
template <int L, int V, bool XF32, bool RF32>
__global__ __launch_bounds__(RowShape<L>::kThreads) void add_rmsnorm_kernel(NormArgs a)
{
#pragma clang fp contract(off)
    constexpr int ROWS = RowShape<L>::kRows;
    __shared__ RowParts<L> parts;
    const int tid = threadIdx.x, li = tid % L;
    const int H = a.H;
    for (int64_t m = (int64_t)blockIdx.x * ROWS + tid / L; m < a.M; m += (int64_t)gridDim.x * ROWS) {
        const size_t base = (size_t)m * H;
        auto count = [&](int i) { return min(8, H - (li + i * L) * 8); };
        float t[V][8];
        double ss = 0.0;
        uint32_t top = 0;
        {
            Raw8<XF32> x[V];
            Raw8<RF32> r[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (count(i) > 0) x[i] = load8<XF32>(a.x, base + (li + i * L) * 8, count(i));
            if (a.residual != nullptr) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (count(i) > 0) r[i] = load8<RF32>(a.residual, base + (li + i * L) * 8, count(i));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int n = count(i);
                if (n <= 0) continue;
                const size_t at = (size_t)(li + i * L) * 8;
                float w[8];
                if (a.w_type == kTypeF32) {
                    const Raw8<true> raw = load8<true>(a.weight, at, n);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = raw.get(j);
                } else {
                    const Raw8<false> raw = load8<false>(a.weight, at, n);
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = raw.get(j);
                }
                Raw8<RF32> out;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = x[i].get(j);
                    if (a.residual != nullptr) v = r[i].get(j) + v;
                    if constexpr (!RF32) v = round_to_bf16(v);
                    out.set(j, v);
                    ss += (double)v * (double)v;
                    t[i][j] = v * w[j];
                    top = max(top, __float_as_uint(t[i][j]) & 0x7FFFFFFFu);
                }
                if (a.residual_out != nullptr) store8<RF32>(a.residual_out, base + at, n, out);
            }
        }
        reduce_row<L>(ss, top, parts);
        const float rstd = (float)(1.0 / sqrt(ss / (double)H + a.eps));
        const float amax = round_to_bf16(__uint_as_float(top) * rstd);
        const QuantScale qs = a.q_type == kQuantInt8 ? int8_scale(amax) : quant_scale(amax);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int n = count(i);
            if (n <= 0) continue;
            const size_t at = base + (size_t)(li + i * L) * 8;
            Raw8<false> y;
#pragma unroll
            for (int j = 0; j < 8; ++j) y.set(j, round_to_bf16(t[i][j] * rstd));
            if (a.y != nullptr) store8<false>(a.y, at, n, y);
            if (a.q_type == kQuantNone) continue;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = quant_div(y.get(j), qs);
            store_codes(a.q, at, n, encode8(v, a.q_type));
        }
        if (a.q_type != kQuantNone && li == 0) a.scale[m] = qs.s;
    }
}

// int8 codes and scales of the rows of a bf16 matrix, laid out over threads as
// above.
template <int L, int V>
__global__ __launch_bounds__(RowShape<L>::kThreads) void int8_quantize_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                              int cols, uint8_t* __restrict__ q,
                                                                              float* __restrict__ scale)
{
    __shared__ RowParts<L> parts;
    const int li = threadIdx.x % L;
    for (int64_t m = (int64_t)blockIdx.x * RowShape<L>::kRows + threadIdx.x / L; m < rows;
         m += (int64_t)gridDim.x * RowShape<L>::kRows) {
        const size_t base = (size_t)m * cols;
        auto count = [&](int i) { return min(8, cols - (li + i * L) * 8); };
        Raw8<false> r[V];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (count(i) > 0) r[i] = load8<false>(x, base + (size_t)(li + i * L) * 8, count(i));
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (count(i) > 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(r[i].get(j)) & 0x7FFFFFFFu);
        double none = 0.0;
        reduce_row<L>(none, top, parts);
        const QuantScale qs = int8_scale(__uint_as_float(top));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (count(i) <= 0) continue;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = quant_div(r[i].get(j), qs);
            store_codes(q, base + (size_t)(li + i * L) * 8, count(i), encode8(v, kQuantInt8));
        }
        if (li == 0) scale[m] = qs.s;
    }
}

// Rows beyond what a workgroup's registers hold: one wave a row, read twice.
__global__ __launch_bounds__(256) void int8_quantize_long_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scale)
{
    const int lane = threadIdx.x & 63;
    for (int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); m < rows; m += (int64_t)gridDim.x * 4) {
        const uint16_t* src = x + (size_t)m * cols;
        uint32_t top = 0;
        for (int64_t i = lane; i < cols; i += kWave) top = max(top, (uint32_t)src[i] & 0x7FFFu);
        const QuantScale qs = int8_scale(bf16_bits_to_f32(wave_max_u32(top)));
        for (int64_t i = lane; i < cols; i += kWave)
            q[(size_t)m * cols + i] = (uint8_t)int8_encode(quant_div(bf16_bits_to_f32(src[i]), qs));
        if (lane == 0) scale[m] = qs.s;
    }
}

}  // namespace moe
