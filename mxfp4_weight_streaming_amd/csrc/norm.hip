// norm.hip -- host launchers of the kernels in norm_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "around_choice.hpp"
#include "moe_internal.hpp"
#include "norm_kernels.hpp"

namespace moe {

namespace {

// Workgroups of a launch that strides over its rows: enough for any chip, and
// far below the grid's limit.
constexpr int64_t kMaxGrid = 1 << 20;

template <int L>
dim3 row_grid(int64_t rows)
{
    return dim3((unsigned)std::min<int64_t>((rows + RowShape<L>::kRows - 1) / RowShape<L>::kRows, kMaxGrid));
}

template <int L, int V>
hipError_t norm(const NormArgs& a, hipStream_t s)
{
    const dim3 grid = row_grid<L>(a.M), block(RowShape<L>::kThreads);
    const bool x = a.x_type == kTypeF32, r = a.r_type == kTypeF32;
    if (x && r) hipLaunchKernelGGL((add_rmsnorm_kernel<L, V, true, true>), grid, block, 0, s, a);
    else if (x) hipLaunchKernelGGL((add_rmsnorm_kernel<L, V, true, false>), grid, block, 0, s, a);
    else if (r) hipLaunchKernelGGL((add_rmsnorm_kernel<L, V, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((add_rmsnorm_kernel<L, V, false, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int L, int V>
hipError_t quantise(const uint16_t* x, int64_t rows, int cols, uint8_t* q, float* scale, hipStream_t s)
{
    hipLaunchKernelGGL((int8_quantize_kernel<L, V>), row_grid<L>(rows), dim3(RowShape<L>::kThreads), 0, s, x, rows, cols,
                       q, scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s)
{
    switch (norm_variant(a.M, a.H)) {
        case kNorm16x1: return norm<16, 1>(a, s);
        case kNorm16x2: return norm<16, 2>(a, s);
        case kNorm64x1: return norm<64, 1>(a, s);
        case kNorm64x2: return norm<64, 2>(a, s);
        case kNorm256x1: return norm<256, 1>(a, s);
        case kNorm512x1: return norm<512, 1>(a, s);
        case kNorm512x2: return norm<512, 2>(a, s);
        case kNorm512x4: return norm<512, 4>(a, s);
        default: return norm<512, 8>(a, s);
    }
}

hipError_t launch_int8_quantize(const uint16_t* x, int rows, int cols, uint8_t* q, float* scale, hipStream_t s)
{
    switch (quant_variant(rows, cols)) {
        case kQuant16x1: return quantise<16, 1>(x, rows, cols, q, scale, s);
        case kQuant64x1: return quantise<64, 1>(x, rows, cols, q, scale, s);
        case kQuant64x2: return quantise<64, 2>(x, rows, cols, q, scale, s);
        case kQuant512x1: return quantise<512, 1>(x, rows, cols, q, scale, s);
        case kQuant512x4: return quantise<512, 4>(x, rows, cols, q, scale, s);
        default: break;
    }
    hipLaunchKernelGGL(int8_quantize_long_kernel, row_grid<64>(rows), dim3(256), 0, s, x, (int64_t)rows, cols, q, scale);
    return hipGetLastError();
}

}  // namespace moe
