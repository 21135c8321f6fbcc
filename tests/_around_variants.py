"""Sizes that reach every kernel variant of the norm, the int8 quantiser and the
int8 product: run by tests/test_gpu_around_variants.py, and held to reach them
all by tests/test_around_variants.py."""

# rows x elements: around each bound of the row kernels, few and many rows
NORM = ([(M, H) for M in (2047, 2048, 2049) for H in (513, 1000, 1001, 1024)] +
        [(3, 128), (3, 129), (3, 256), (3, 257), (3, 512), (3, 513), (3, 2048), (3, 2049), (3, 4096), (3, 4097),
         (3, 8192), (3, 8193), (3, 16384), (3, 16385), (5, 32768)])
QUANT = ([(M, H) for M in (2047, 2048, 2051) for H in (512, 513, 1001, 1024, 1025)] +
         [(3, 128), (3, 129), (3, 4096), (3, 4097), (3, 8203), (3, 16384), (3, 16385), (3, 40000)])

# tokens x channels of each tile, with whole tiles only and with odd remainders, by
# the tile's step and ring
INT8_TILES = {
    "256x256": ((64, 4), [(768, 20480), (513, 20003)]),
    "128x128": ((128, 2), [(1024, 4096), (777, 4099)]),
    "128x64": ((128, 2), [(512, 4096), (300, 5121)]),
    "64x128": ((128, 3), [(64, 32768), (129, 20003)]),
    "64x64": ((128, 3), [(256, 4096), (300, 8193)]),
    "32x64": ((128, 4), [(32, 12288), (33, 4099)]),
    "32x32": ((128, 4), [(64, 512), (65, 515)]),
}
# tokens x channels of each GEMV
INT8_GEMV = {
    "64 lanes": [(1, 8191), (2, 2560), (3, 33), (4, 8191)],
    "16 lanes": [(1, 8192), (2, 20000), (3, 8193), (4, 65535)],
    "16 lanes, two channels": [(1, 65536), (2, 65537), (3, 70001), (4, 65551)],
}
GEMV_DEPTHS = (1, 15, 16, 17, 256, 511, 512, 640, 769, 1280, 1281, 2560, 2576, 4999, 5120)


def tile_depths(step, ring):
    """Depths K around the ring's length: none, one, ring - 1 .. ring + 2 whole steps, an odd and an even count beyond,
    alone and with a part step behind them; and rows that are no multiple of 16 codes."""
    counts = sorted({1, 2, ring - 1, ring, ring + 1, ring + 2, 2 * ring + 1, 2 * ring + 2})
    whole = [n * step for n in counts]
    part = [n * step + more for n, more in zip([0] + counts, (16, 16, 48, step - 16, 32, 16, step - 16, 48, 32))]
    odd = [15, step - 1, step + 1, 2 * step + 4, 3 * step - 3, (ring + 1) * step + 7, 6 * step + 33]
    return whole + part + odd


def int8_sizes():
    """Every (M, N, K) of the int8 product's cases."""
    for (step, ring), sizes in INT8_TILES.values():
        for M, N in sizes:
            yield from ((M, N, K) for K in tile_depths(step, ring))
    for sizes in INT8_GEMV.values():
        for M, N in sizes:
            yield from ((M, N, K) for K in GEMV_DEPTHS)
