// lora_common.hpp -- low-rank adapters of many requests (gfx950), what their
// kernels and the int8 product's share: token m has adapter i = ids[m], and
//   u[m] = scale[i] A[i] x[m]             (r values, fp32; kept with zeros behind
//                                          them up to a multiple of 32, rp)
//   out[m] = round(base[m] + B[i] u[m])   base alone where i is no adapter
//
// Tokens are taken as they stand, 16 at a time, which is a matrix instruction's
// width: a request's tokens follow one another, so 16 of them have few adapters.
// Each adapter among them is multiplied by all 16, and each token takes its own
// adapter's result, so nothing of another adapter, infinities and NaN included,
// reaches it.  Where tiles are few, their adapters are dealt to several
// workgroups (slots).
//
// v_mfma_f32_16x16x32_bf16: lane l gives row l % 16, values 8 (l / 16).. of both
// operands, and gets rows 4 (l / 16) + 0..3 of the first and row l % 16 of the
// second, the token.  u goes into the second product as three bf16 numbers that
// add up to the fp32 one (8 bits each), so it is not rounded.
#pragma once

#include "around_common.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_half __attribute__((aligned(2)));    // at any bf16
typedef u32x2 u32x2_half __attribute__((aligned(2)));
typedef f32x4 f32x4_word __attribute__((aligned(4)));    // at any fp32

// The adapter of token m, or -1; -2 for what is no token.
__device__ __forceinline__ int adapter_of(const LoraArgs& g, int64_t m)
{
    if (m >= g.M) return -2;
    const int i = g.ids[m];
    return i >= 0 && i < g.L ? i : -1;
}

// Calls f(adapter, mask of the tokens that have it) for each adapter among the
// wave's 16 tokens (-1, none, too) that falls to `slot` of `slots` (a power of
// two).
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int slot, int slots, F f)
{
    uint32_t todo = (uint32_t)__ballot(id >= -1) & 0xFFFFu;
    for (int d = 0; todo != 0; ++d) {
        const int i = __builtin_amdgcn_readlane(id, (int)__builtin_ctz(todo));
        const uint32_t mask = (uint32_t)__ballot(id == i) & 0xFFFFu;
        todo &= ~mask;
        if ((d & (slots - 1)) == slot) f(i, mask);
    }
}

// Values k .. k + 7 of a row of n, zeros behind it.  EVEN: n is a multiple of 8,
// so they are all there or none is, and the load needs no branch.
template <bool EVEN>
__device__ __forceinline__ u32x4 load_bf16x8(const uint16_t* row, int k, int n)
{
    if constexpr (EVEN) {
        const u32x4 v = *reinterpret_cast<const u32x4_half*>(row + (k < n ? k : 0));
        return k < n ? v : u32x4{0, 0, 0, 0};
    }
    const uint16_t* p = row + k;
    if (k + 8 <= n) return *reinterpret_cast<const u32x4_half*>(p);
    uint32_t d[4] = {0, 0, 0, 0};
    if (k < n)
#pragma unroll
        for (int i = 0; i < 7; ++i) {                    // (all asked for at once)
            const uint32_t v = p[min(i, n - 1 - k)];
            d[i >> 1] |= (k + i < n ? v : 0) << (16 * (i & 1));
        }
    return u32x4{d[0], d[1], d[2], d[3]};
}

// acc + the sum of 8 products, one after another in fp32.
__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float acc)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        acc = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), acc);
        acc = fmaf(__uint_as_float(a[e] & 0xFFFF0000u), __uint_as_float(b[e] & 0xFFFF0000u), acc);
    }
    return acc;
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two fp32 values as three pairs of bf16 that add up to them.
struct Split3 {
    uint32_t v[3];
};

__device__ __forceinline__ Split3 split_pair(float a, float b)
{
    Split3 s;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        const uint32_t lo = f32_to_bf16_bits(a), hi = f32_to_bf16_bits(b);
        s.v[p] = lo | hi << 16;
        a -= bf16_bits_to_f32(lo);
        b -= bf16_bits_to_f32(hi);
    }
    return s;
}

}  // namespace moe
