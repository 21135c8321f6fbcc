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
    const LoraPlan p = lora_plan(a.M, a.N, a.r);
    a.slots = p.expand_slots;
    a.token_tiles = p.token_tiles;
    const int64_t grid = ceil_div(a.M, 16 * p.token_tiles) * ceil_div(a.N, 256) * a.slots;
    if (grid * 256 > kMaxThreads) return hipErrorInvalidConfiguration;
    const auto kernel = a.r % 8 == 0 ? lora_expand_kernel<F32, RK, true> : lora_expand_kernel<F32, RK, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <bool F32>
hipError_t expand_ranks(const LoraArgs& a, hipStream_t s)
{
    return a.r <= 32 ? expand<F32, 1>(a, s) : a.r <= 64 ? expand<F32, 2>(a, s) : expand<F32, 4>(a, s);
}

}  // namespace

hipError_t launch_lora_shrink(LoraArgs a, hipStream_t s)
{
    a.slots = lora_plan(a.M, a.N, a.r).shrink_slots;
    const int64_t grid = ceil_div(a.M, 16) * (a.rp / 16) * a.slots;
    if (grid * 512 > kMaxThreads) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(lora_shrink_kernel, dim3((unsigned)grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s)
{
    const hipError_t e = launch_lora_shrink(a, s);
    if (e != hipSuccess) return e;
    return a.out_type == kTypeF32 ? expand_ranks<true>(a, s) : expand_ranks<false>(a, s);
}

}  // namespace moe
