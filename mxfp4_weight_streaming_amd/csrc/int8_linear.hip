// int8_linear.hip -- host launchers of the kernels in int8_kernels.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "int8_kernels.hpp"
#include "moe_internal.hpp"

namespace moe {

namespace {

constexpr int kCus = 256;      // compute units

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

// Whether the token rows, padded to steps of `step` codes, fit the GEMV's LDS.
bool gemv_fits(const Int8Args& a, int step) { return a.M <= kInt8GemvTokens && a.M * ceil_div(a.K, step) * step <= kInt8GemvLds; }

template <int BM, int BN, int WM, int WN, int BK, int S, int EU>
hipError_t tiles(Int8Args a, hipStream_t s)
{
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

// The tile shapes, and what a tile takes on a compute unit that always has
// others to overlap it with: us per 128 codes of K, from products of
// 512 x 157184 x 2560.
struct TileShape {
    int bm, bn;
    double cost;
};
constexpr TileShape kTiles[] = {{256, 256, 2.78}, {128, 128, 0.89}, {128, 64, 0.50}, {64, 128, 0.55},
                                {64, 64, 0.31},   {32, 64, 0.17},   {32, 32, 0.12}};

// Large tiles move the fewest bytes a product, small ones fill the chip when
// there are few: each shape's time is its cost times the tiles a compute unit
// gets, between the mean and the most (the busiest unit overlaps its tiles).
// Measured against the best of a sweep at 22 sizes from 8 x 1536 x 768 to
// 512 x 157184 x 2560: within 10% of it at each.
int best_tile(int64_t M, int64_t N)
{
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        const int64_t tiles = ceil_div(M, kTiles[i].bm) * ceil_div(N, kTiles[i].bn);
        const double t = kTiles[i].cost * std::max(1.0, ((double)tiles / kCus + (double)ceil_div(tiles, kCus)) / 2);
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best;
}

}  // namespace

hipError_t launch_int8_linear(const Int8Args& a, hipStream_t s)
{
    // Up to 4 tokens the dot instructions keep up with the memory and a wave
    // reads whole rows; from 5 tokens on the matrix cores are faster
    // (157,184 x 2,560: 4 tokens 65.0 us against 72.2 us, 8 tokens 88.2
    // against 74.9).  Few channels are split over all lanes of a wave, so that
    // every compute unit has some (1,536 x 2,560, 4 tokens: 5.2 us against 6.5
    // with 16 lanes); many are taken two a lane, which reads the tokens from
    // LDS half as often (157,184 x 2,560, 4 tokens: 65.0 us against 67.8).
    if (a.N < 8192) {
        if (gemv_fits(a, 3 * 1024)) return gemv_tokens<3, 64, 1>(a, s);
    } else if (a.N < 65536) {
        if (gemv_fits(a, 5 * 256)) return gemv_tokens<5, 16, 1>(a, s);
    } else {
        if (gemv_fits(a, 2 * 256)) return gemv_tokens<2, 16, 2>(a, s);
    }
    hipError_t e = hipErrorInvalidConfiguration;
    switch (best_tile(a.M, a.N)) {
        case 0: break;
        case 1: e = tiles<128, 128, 2, 2, 128, 2, 2>(a, s); break;
        case 2: e = tiles<128, 64, 2, 2, 128, 2, 3>(a, s); break;
        case 3: e = tiles<64, 128, 2, 2, 128, 3, 3>(a, s); break;
        case 4: e = tiles<64, 64, 2, 2, 128, 3, 3>(a, s); break;
        case 5: e = tiles<32, 64, 1, 4, 128, 4, 3>(a, s); break;
        default: e = tiles<32, 32, 1, 2, 128, 4, 2>(a, s); break;
    }
    // the largest tiles are also what is left when there are too many smaller ones
    return e == hipErrorInvalidConfiguration ? tiles<256, 256, 2, 4, 64, 4, 2>(a, s) : e;
}

}  // namespace moe
