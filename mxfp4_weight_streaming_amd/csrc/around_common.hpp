// around_common.hpp -- device helpers shared by the operators around the expert
// layer (gfx950).
#pragma once

#include "around_types.hpp"
#include "device_common.hpp"

namespace moe {

__device__ __forceinline__ uint32_t f32_to_bf16_bits(float v)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);   // round to nearest even
}

__device__ __forceinline__ float round_to_bf16(float v) { return bf16_bits_to_f32(f32_to_bf16_bits(v)); }

__device__ __forceinline__ float load_typed(const void* p, int type, size_t i)
{
    return type == kTypeF32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v)
{
    return __builtin_bit_cast(double, dpp_u64<CTRL>(__builtin_bit_cast(uint64_t, v)));
}

__device__ __forceinline__ double row_lane_f64(double v, int lane)
{
    return __builtin_bit_cast(double, read_lane_u64(__builtin_bit_cast(uint64_t, v), lane));
}

// Sum over each row of 16 lanes, and over the wave, in a fixed order; every lane
// gets it.
__device__ __forceinline__ double row_sum_f64(double v)
{
    v += dpp_f64<kDppXor1>(v);
    v += dpp_f64<kDppXor2>(v);
    v += dpp_f64<kDppHalfMirror>(v);
    return v + dpp_f64<kDppMirror>(v);
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
    v = row_sum_f64(v);
    return (row_lane_f64(v, 0) + row_lane_f64(v, 16)) + (row_lane_f64(v, 32) + row_lane_f64(v, 48));
}

// Largest unsigned value of each row of 16 lanes.
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v)
{
    v = max(v, dpp_u32<kDppXor1>(v));
    v = max(v, dpp_u32<kDppXor2>(v));
    v = max(v, dpp_u32<kDppHalfMirror>(v));
    return max(v, dpp_u32<kDppMirror>(v));
}

}  // namespace moe
