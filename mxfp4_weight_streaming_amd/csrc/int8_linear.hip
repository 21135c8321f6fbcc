// int8_linear.hip -- host launchers of the kernels in int8_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "around_choice.hpp"
#include "int8_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

namespace {

template <int MT, int U, int L, int R>
hipError_t gemv(const Int8Args& a, hipStream_t s)
{
    const int64_t blocks = ceil_div(a.N, 4 * R * (64 / L)), padded = ceil_div(ceil_div(a.K, 16), L * U) * L * U;
    hipLaunchKernelGGL((int8_gemv_kernel<MT, U, L, R>), dim3((unsigned)std::min<int64_t>(blocks, 8 * kCus)), dim3(256),
                       (uint32_t)(a.M * padded * 16), s, a);
    return hipGetLastError();
}

template <int U, int L, int R>
hipError_t gemv_tokens(const Int8Args& a, hipStream_t s)
{
    if (a.M == 1) return gemv<1, U, L, R>(a, s);
    if (a.M == 2) return gemv<2, U, L, R>(a, s);
    return gemv<4, U, L, R>(a, s);
}

template <Int8Variant V, int WM, int WN, int EU>
hipError_t tiles(Int8Args a, hipStream_t s)
{
    constexpr int BM = kTileShapes[V].bm, BN = kTileShapes[V].bn, BK = kTileShapes[V].bk, S = kTileShapes[V].ring;
    constexpr size_t lds = (size_t)S * (BM + BN) * BK;
    // the split of the tiles over the XCDs: the fewest tiles on any XCD, then
    // the fewest rows read by one (4096 x 4096 x 2560: 47.8 us with every XCD
    // reading all tokens, 46.1 us with the split chosen here)
    const int64_t mt = ceil_div(a.M, BM), nt = ceil_div(a.N, BN);
    int64_t most = 0, rows = 0;
    for (int xm = 1; xm <= 8; xm *= 2) {
        const int64_t mx = ceil_div(mt, xm), nx = ceil_div(nt, 8 / xm), r = mx * BM + nx * BN;
        if (xm == 1 || mx * nx < most || (mx * nx == most && r < rows)) {
            a.xm = xm;
            most = mx * nx;
            rows = r;
        }
    }
    const int64_t grid = most * 8;
    if (grid * 64 * WM * WN > 0xFFFFFFFFll) return hipErrorInvalidConfiguration;   // beyond a launch's threads
    const auto kernel = a.K % 16 == 0 ? int8_tile_kernel<BM, BN, WM, WN, BK, S, EU, true>
                                      : int8_tile_kernel<BM, BN, WM, WN, BK, S, EU, false>;
    if (lds > 64 * 1024) {   // above the default dynamic-LDS limit
        const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * WM * WN), (uint32_t)lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_linear(const Int8Args& a, hipStream_t s)
{
    hipError_t e = hipErrorInvalidConfiguration;
    switch (int8_variant(a.M, a.N, a.K)) {
        case kGemv64Lanes: return gemv_tokens<3, 64, 1>(a, s);
        case kGemv16Lanes: return gemv_tokens<5, 16, 1>(a, s);
        case kGemv16LanesPairs: return gemv_tokens<2, 16, 2>(a, s);
        case kTile128x128: e = tiles<kTile128x128, 2, 2, 2>(a, s); break;
        case kTile128x64: e = tiles<kTile128x64, 2, 2, 3>(a, s); break;
        case kTile64x128: e = tiles<kTile64x128, 2, 2, 3>(a, s); break;
        case kTile64x64: e = tiles<kTile64x64, 2, 2, 3>(a, s); break;
        case kTile32x64: e = tiles<kTile32x64, 1, 4, 3>(a, s); break;
        case kTile32x32: e = tiles<kTile32x32, 1, 2, 2>(a, s); break;
        default: break;
    }
    // the largest tiles are also what is left when there are too many smaller ones
    return e == hipErrorInvalidConfiguration ? tiles<kTile256x256, 2, 4, 2>(a, s) : e;
}

}  // namespace moe
