// lora.hip -- host launchers of the kernels in lora_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "around_choice.hpp"
#include "lora_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

size_t lora_workspace(int64_t M, int64_t N, int r) { return align256((size_t)M * r * 4) + (size_t)M * N * 4; }

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t s)
{
    const auto grid = [](int64_t blocks) { return dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)); };
    hipLaunchKernelGGL(lora_shrink_kernel, grid(ceil_div(a.M * a.r, 4)), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lora_expand_kernel, grid(ceil_div(a.M * a.N, 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_int8_linear_lora(const Int8Args& p, LoraArgs a, hipStream_t s)
{
    Int8Args g = p;
    g.out = reinterpret_cast<uint8_t*>(a.u) + align256((size_t)a.M * a.r * 4);
    g.out_type = kTypeF32;
    const hipError_t e = launch_int8_linear(g, s);
    if (e != hipSuccess) return e;
    a.base = g.out;
    a.base_type = kTypeF32;
    return launch_lora_add(a, s);
}

}  // namespace moe
