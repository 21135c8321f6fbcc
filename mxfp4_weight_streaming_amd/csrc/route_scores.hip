// route_scores.hip -- host launcher of the kernel in score_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "moe_internal.hpp"
#include "score_kernels.hpp"

namespace moe {

hipError_t launch_route_scores(const ScoreArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)std::min<int64_t>((a.M + 3) / 4, (int64_t)1 << 20));
    hipLaunchKernelGGL(route_scores_kernel, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
