// lora.hip -- host launchers of the kernels in lora_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "beside_choice.hpp"
#include "lora_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

size_t lora_workspace(int64_t M, int r) { return align256((size_t)M * lora_padded(r) * 4); }

namespace {

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;   // of a launch

template <bool F32, int RK>
hipError_t expand(LoraArgs a, hipStream_t s)
{
    const LoraPlan p = lora_plan(a.M, a.N, a.K, a.r);
    a.slots = p.expand_slots;
    a.token_tiles = p.token_tiles;
    const int64_t grid = ceil_div(a.M, 16 * p.token_tiles) * ceil_div(a.N, 256) * a.slots;
    if (grid * 256 > kMaxThreads) return hipErrorInvalidConfiguration;
    const auto kernel = a.r % 8 == 0 ? lora_expand_kernel<F32, RK, true> : lora_expand_kernel<F32, RK, false>;
    const uint32_t lds = 3 * 16 * p.token_tiles * (a.rp / 2 + 4) * 4;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), lds, s, a);
    return hipGetLastError();
}

template <bool F32>
hipError_t expand_ranks(const LoraArgs& a, hipStream_t s)
{
    return a.r <= 32 ? expand<F32, 1>(a, s) : a.r <= 64 ? expand<F32, 2>(a, s) : expand<F32, 4>(a, s);
}

}  // namespace

namespace {

template <bool F32, bool FUSED>
hipError_t few(const LoraArgs& a, hipStream_t s)
{
    const auto kernel = a.r % 8 == 0 ? lora_few_kernel<F32, FUSED, true> : lora_few_kernel<F32, FUSED, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(a.M * ceil_div(a.N, 256))), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_shrink(LoraArgs a, hipStream_t s)
{
    const LoraPlan p = lora_plan(a.M, a.N, a.K, a.r);
    if (p.shrink_few) {
        const auto kernel = a.K % 8 == 0 ? lora_shrink_few_kernel<true> : lora_shrink_few_kernel<false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.M * ceil_div(a.r, 16))), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    a.slots = p.shrink_slots;
    const int rr = a.r > 16 ? 2 : 1;
    const int64_t grid = ceil_div(a.M, 16) * ceil_div(a.r, 16 * rr) * a.slots;
    if (grid * 512 > kMaxThreads) return hipErrorInvalidConfiguration;
    const auto kernel = rr == 2 ? lora_shrink_kernel<2> : lora_shrink_kernel<1>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s)
{
    const LoraPlan p = lora_plan(a.M, a.N, a.K, a.r);
    const bool f32 = a.out_type == kTypeF32;
    if (p.few && p.fused) return f32 ? few<true, true>(a, s) : few<false, true>(a, s);
    const hipError_t e = launch_lora_shrink(a, s);
    if (e != hipSuccess) return e;
    if (p.few) return f32 ? few<true, false>(a, s) : few<false, false>(a, s);
    return f32 ? expand_ranks<true>(a, s) : expand_ranks<false>(a, s);
}

}  // namespace moe
