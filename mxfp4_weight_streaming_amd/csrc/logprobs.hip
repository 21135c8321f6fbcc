// logprobs.hip -- host launchers of the kernels in logprob_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "logprob_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

size_t logprob_workspace(int64_t, int, int) { return 0; }

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL(logprob_row_kernel, dim3((unsigned)std::min<int64_t>(a.M, 1 << 20)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
