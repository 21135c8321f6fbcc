// around_choice.hpp -- which variant of their kernels the norm, the int8
// quantiser and the int8 product run, by sizes alone.  Plain C++: a host
// program asks the same rules which variants a set of sizes reaches.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- rows: L threads a row, V vectors of 8 elements a thread ------------------
// Few rows are a chain of latencies: more threads a row shorten it.  Many rows
// are bound by bytes: fewer threads waste fewer lanes and need no barrier
// (1,000 elements: 301 rows 4.9 us with a wave a row, 4.3 with 256 threads;
// 16,384 rows 33.3 against 36.4).
constexpr bool few_rows(int64_t rows) { return rows < 2048; }

enum NormVariant {
    kNorm16x1, kNorm16x2, kNorm64x1, kNorm64x2, kNorm256x1, kNorm512x1, kNorm512x2, kNorm512x4, kNorm512x8, kNormVariants
};

constexpr NormVariant norm_variant(int64_t M, int H)
{
    const int64_t vecs = ceil_div(H, 8);
    if (vecs <= 16) return kNorm16x1;
    if (vecs <= 32) return kNorm16x2;
    if (vecs <= 64) return kNorm64x1;
    if (vecs <= 128 && !few_rows(M)) return kNorm64x2;
    if (vecs <= 256) return kNorm256x1;
    if (vecs <= 512) return kNorm512x1;
    if (vecs <= 1024) return kNorm512x2;
    if (vecs <= 2048) return kNorm512x4;
    return kNorm512x8;
}

enum QuantVariant { kQuant16x1, kQuant64x1, kQuant64x2, kQuant512x1, kQuant512x4, kQuantLong, kQuantVariants };

constexpr QuantVariant quant_variant(int64_t rows, int64_t cols)
{
    const int64_t vecs = ceil_div(cols, 8);
    if (vecs <= 16) return kQuant16x1;
    if (vecs <= 64) return kQuant64x1;
    if (vecs <= 128 && !few_rows(rows)) return kQuant64x2;
    if (vecs <= 512) return kQuant512x1;
    if (vecs <= 2048) return kQuant512x4;
    return kQuantLong;
}

// ---- int8 product --------------------------------------------------------------
constexpr int kCus = 256;                  // compute units
constexpr int kInt8GemvTokens = 4;
constexpr int64_t kInt8GemvLds = 64 * 1024;

enum Int8Variant {
    kTile256x256, kTile128x128, kTile128x64, kTile64x128, kTile64x64, kTile32x64, kTile32x32, kTiles,
    kGemv64Lanes = kTiles, kGemv16Lanes, kGemv16LanesPairs, kInt8Variants
};

// The tiles: tokens, channels, codes of K a step, steps in the ring; and what a
// tile takes on a compute unit that always has others to overlap it with: us per
// 128 codes of K, from products of 512 x 157184 x 2560.
struct TileShape {
    int bm, bn, bk, ring;
    double cost;
};
constexpr TileShape kTileShapes[kTiles] = {{256, 256, 64, 4, 2.78}, {128, 128, 128, 2, 0.89}, {128, 64, 128, 2, 0.50},
                                           {64, 128, 128, 3, 0.55}, {64, 64, 128, 3, 0.31},   {32, 64, 128, 4, 0.17},
                                           {32, 32, 128, 4, 0.12}};

// Large tiles move the fewest bytes a product, small ones fill the chip when
// there are few: each shape's time is its cost times the tiles a compute unit
// gets, between the mean and the most (the busiest unit overlaps its tiles).
// Measured against the best of the seven at 22 sizes from 8 x 1536 x 768 to
// 512 x 157184 x 2560: within 6% of it at 17, and 17 to 19% above it at five
// with 2.5 to 10 tiles of 64 x 64 a compute unit, where a size smaller than the
// one chosen is faster (512 x 5120 x 2560: 18.7 us with 128 x 64, 15.8 with
// 64 x 64).
constexpr Int8Variant int8_tile(int64_t M, int64_t N)
{
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < kTiles; ++i) {
        const int64_t tiles = ceil_div(M, kTileShapes[i].bm) * ceil_div(N, kTileShapes[i].bn);
        const double t = kTileShapes[i].cost * std::max(1.0, ((double)tiles / kCus + (double)ceil_div(tiles, kCus)) / 2);
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return (Int8Variant)best;
}

// Whether the token rows, padded to steps of `step` codes, fit the GEMV's LDS.
constexpr bool gemv_fits(int64_t M, int64_t K, int step)
{
    return M <= kInt8GemvTokens && M * ceil_div(K, step) * step <= kInt8GemvLds;
}

// Up to 4 tokens the dot instructions keep up with the memory and a wave
// reads whole rows; from 5 tokens on the matrix cores are faster
// (157,184 x 2,560: 4 tokens 65.0 us against 72.2 us, 8 tokens 88.2
// against 74.9).  Few channels are split over all lanes of a wave, so that
// every compute unit has some (1,536 x 2,560, 4 tokens: 5.2 us against 6.5
// with 16 lanes); many are taken two a lane, which reads the tokens from
// LDS half as often (157,184 x 2,560, 4 tokens: 65.0 us against 67.8).
constexpr Int8Variant int8_variant(int64_t M, int64_t N, int64_t K)
{
    if (N < 8192) {
        if (gemv_fits(M, K, 3 * 1024)) return kGemv64Lanes;
    } else if (N < 65536) {
        if (gemv_fits(M, K, 5 * 256)) return kGemv16Lanes;
    } else {
        if (gemv_fits(M, K, 2 * 256)) return kGemv16LanesPairs;
    }
    return int8_tile(M, N);
}

}  // namespace moe
