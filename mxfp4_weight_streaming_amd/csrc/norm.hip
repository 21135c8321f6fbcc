// norm.hip -- host launchers of the kernels in norm_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "moe_internal.hpp"
#include "norm_kernels.hpp"

namespace moe {

// Workgroups of a launch that strides over its work: enough for any chip, and
// far below the grid's limit.
constexpr int64_t kMaxGrid = 1 << 20;

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s)
{
    const size_t lds = (size_t)a.H * 4;
    if (lds > 64 * 1024) {   // above the default dynamic-LDS limit
        const hipError_t e = hipFuncSetAttribute((const void*)add_rmsnorm_kernel,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)std::min<int64_t>(a.M, kMaxGrid));
    hipLaunchKernelGGL(add_rmsnorm_kernel, grid, dim3(kNormThreads), (uint32_t)lds, s, a);
    return hipGetLastError();
}

hipError_t launch_int8_quantize(const uint16_t* x, int rows, int cols, uint8_t* q, float* scale, hipStream_t s)
{
    const dim3 grid((unsigned)std::min<int64_t>(((int64_t)rows + 3) / 4, kMaxGrid));
    hipLaunchKernelGGL(int8_quantize_kernel, grid, dim3(256), 0, s, x, (int64_t)rows, cols, q, scale);
    return hipGetLastError();
}

}  // namespace moe
