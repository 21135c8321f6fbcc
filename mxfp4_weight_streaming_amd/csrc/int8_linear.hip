// int8_linear.hip -- host launcher of the kernels in int8_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "int8_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

hipError_t launch_int8_linear(const Int8Args& a, hipStream_t s)
{
    const int64_t tiles = ((a.M + kInt8Tile - 1) / kInt8Tile) * ((a.N + kInt8Tile - 1) / kInt8Tile);
    const dim3 grid((unsigned)std::min<int64_t>(tiles, (int64_t)1 << 20));
    hipLaunchKernelGGL(int8_linear_kernel, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
