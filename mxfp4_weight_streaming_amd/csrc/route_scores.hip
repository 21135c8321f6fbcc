// route_scores.hip -- host launcher of the kernel in score_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "moe_internal.hpp"
#include "score_kernels.hpp"

namespace moe {

hipError_t launch_route_scores(const ScoreArgs& a, hipStream_t s)
{
    // workgroups of 4 waves, one token a wave, each striding over the tokens: as
    // many as the chip holds at once at up to 128 experts or nearly (7 waves a
    // SIMD: 1,792), and twice as many at 512 and sigmoid (4 waves: 1,024)
    const dim3 grid((unsigned)std::min<int64_t>((a.M + 3) / 4, 2048)), block(256);
    const bool softmax = a.score == kScoreSoftmax;
#define MOE_ROUTE_SCORES(PER)                                                                             \
    do {                                                                                                  \
        if (softmax) hipLaunchKernelGGL((route_scores_kernel<PER, true>), grid, block, 0, s, a);          \
        else hipLaunchKernelGGL((route_scores_kernel<PER, false>), grid, block, 0, s, a);                 \
    } while (0)
    if (a.E <= 64) MOE_ROUTE_SCORES(1);
    else if (a.E <= 128) MOE_ROUTE_SCORES(2);
    else if (a.E <= 256) MOE_ROUTE_SCORES(4);
    else MOE_ROUTE_SCORES(8);
#undef MOE_ROUTE_SCORES
    return hipGetLastError();
}

}  // namespace moe
