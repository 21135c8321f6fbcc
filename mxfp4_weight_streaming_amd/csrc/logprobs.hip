// logprobs.hip -- host launchers of the kernels in logprob_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "beside_choice.hpp"
#include "logprob_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

namespace {

size_t maxima_bytes(int64_t M, const LogprobPlan& p) { return align256((size_t)M * p.groups * 256 * 4); }

}  // namespace

size_t logprob_workspace(int64_t M, int V, int topk)
{
    // what serves M rows serves fewer, so the most rows that are split count
    const int64_t rows = std::min<int64_t>(M, kLogprobSplitRows);
    const LogprobPlan p = logprob_plan(1, V);
    if (p.parts == 1) return 0;
    return (topk > 0 ? maxima_bytes(rows, p) : 0) + (size_t)rows * kLogprobMaxParts * sizeof(RowSums);
}

namespace {

template <bool F32, int T>
hipError_t rows(const LogprobArgs& a, hipStream_t s)
{
    const size_t lds = a.topk > 0 ? (size_t)a.groups * T * 4 : 0;
    const auto kernel = logprob_rows_kernel<F32, T>;
    if (lds + sizeof(LogprobLds<T>) > 64 * 1024) {   // above the default limit
        const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(a.M, 1 << 20)), dim3(T), (uint32_t)lds, s, a);
    return hipGetLastError();
}

template <bool F32>
hipError_t launch(LogprobArgs a, hipStream_t s)
{
    const LogprobPlan p = logprob_plan(a.M, a.V);
    a.segments = p.segments;
    a.group_segments = p.group_segments;
    a.groups = p.groups;
    a.parts = p.parts;
    a.part_segments = p.part_segments;
    if (p.threads == 64) {
        const int64_t grid = ceil_div(a.M, a.topk > 0 ? 2 : 4);
        if (grid * 256 > 0xFFFFFFFFll) return hipErrorInvalidConfiguration;   // beyond a launch's threads
        const auto kernel = p.segments == 1 ? logprob_short_kernel<F32, true> : logprob_short_kernel<F32, false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    if (p.parts == 1) return p.threads == 256 ? rows<F32, 256>(a, s) : p.threads == 512 ? rows<F32, 512>(a, s) : rows<F32, 1024>(a, s);
    a.maxima = static_cast<float*>(a.ws);
    a.sums = reinterpret_cast<RowSums*>(static_cast<uint8_t*>(a.ws) + (a.topk > 0 ? maxima_bytes(a.M, p) : 0));
    hipLaunchKernelGGL((logprob_parts_kernel<F32>), dim3((unsigned)(a.M * p.parts)), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((logprob_join_kernel<F32>), dim3((unsigned)a.M), dim3(a.topk > 0 ? kLogprobJoin : 64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s)
{
    return a.type == kTypeF32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
