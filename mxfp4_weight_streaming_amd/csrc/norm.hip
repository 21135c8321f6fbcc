// norm.hip -- host launchers of the kernels in norm_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

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

// Few rows are a chain of latencies: more threads a row shorten it.  Many rows
// are bound by bytes: fewer threads waste fewer lanes and need no barrier
// (1,000 elements: 301 rows 4.9 us with a wave a row, 4.3 with 256 threads;
// 16,384 rows 33.3 against 36.4).
bool few(int64_t rows) { return rows < 2048; }

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s)
{
    const int vecs = (a.H + 7) / 8;
    if (vecs <= 16) return norm<16, 1>(a, s);
    if (vecs <= 32) return norm<16, 2>(a, s);
    if (vecs <= 64) return norm<64, 1>(a, s);
    if (vecs <= 128 && !few(a.M)) return norm<64, 2>(a, s);
    if (vecs <= 256) return norm<256, 1>(a, s);
    if (vecs <= 512) return norm<512, 1>(a, s);
    if (vecs <= 1024) return norm<512, 2>(a, s);
    if (vecs <= 2048) return norm<512, 4>(a, s);
    return norm<512, 8>(a, s);
}

hipError_t launch_int8_quantize(const uint16_t* x, int rows, int cols, uint8_t* q, float* scale, hipStream_t s)
{
    const int64_t vecs = ((int64_t)cols + 7) / 8, n = rows;
    if (vecs <= 16) hipLaunchKernelGGL((int8_quantize_kernel<16, 1>), row_grid<16>(n), dim3(256), 0, s, x, n, cols, q, scale);
    else if (vecs <= 64) hipLaunchKernelGGL((int8_quantize_kernel<64, 1>), row_grid<64>(n), dim3(256), 0, s, x, n, cols, q, scale);
    else if (vecs <= 128 && !few(n)) hipLaunchKernelGGL((int8_quantize_kernel<64, 2>), row_grid<64>(n), dim3(256), 0, s, x, n, cols, q, scale);
    else if (vecs <= 512) hipLaunchKernelGGL((int8_quantize_kernel<512, 1>), row_grid<512>(n), dim3(512), 0, s, x, n, cols, q, scale);
    else if (vecs <= 2048) hipLaunchKernelGGL((int8_quantize_kernel<512, 4>), row_grid<512>(n), dim3(512), 0, s, x, n, cols, q, scale);
    else hipLaunchKernelGGL(int8_quantize_long_kernel, row_grid<64>(n), dim3(256), 0, s, x, n, cols, q, scale);
    return hipGetLastError();
}

}  // namespace moe
