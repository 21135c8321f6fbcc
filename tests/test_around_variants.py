"""CPU-only: the sizes of tests/test_gpu_around_variants.py reach every kernel
variant that the library's rules can choose, and of the int8 tiles every state of
their ring of steps."""
import os
import subprocess

import pytest

from _around_variants import INT8_GEMV, INT8_TILES, GEMV_DEPTHS, NORM, QUANT, int8_sizes, tile_depths

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mxfp4_weight_streaming_amd", "csrc")


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    exe = tmp_path_factory.mktemp("choice") / "around_choice"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "around_choice.cpp")], check=True)

    def run(op, sizes):
        text = "".join(f"{op} {' '.join(map(str, s))}\n" for s in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(list(sizes))
        return got

    return run


def test_row_kernels(choose):
    norms, quants, _ = choose("count", [()])[0]
    assert {v for v, in choose("norm", NORM)} == set(range(norms))
    assert {v for v, in choose("quant", QUANT)} == set(range(quants))


def test_int8_kernels(choose):
    count = choose("count", [()])[0][2]
    assert {g[0] for g in choose("int8", list(int8_sizes()))} == set(range(count))
    # each list is one variant's, in the rules' order: the tiles, then the GEMVs
    for i, (step_ring, sizes) in enumerate(INT8_TILES.values()):
        for M, N in sizes:
            depths = tile_depths(*step_ring)
            got = choose("int8", [(M, N, K) for K in depths])
            assert {(g[0], g[2]) for g in got} == {(i, step_ring[1])}, (M, N)
            step, ring = step_ring
            whole = {g[1] for g, K in zip(got, depths) if K % step == 0}
            assert {1, ring - 1, ring, ring + 1, ring + 2} - {0} <= whole
            direct = {g[1] for g in got if g[3]}
            assert 0 in direct and any(n % 2 for n in direct if n > ring) and any(n % 2 == 0 for n in direct if n > ring)
            assert {0, 1} <= {g[1] for g in got if not g[3]} and any(g[1] > ring for g in got if not g[3])
    for i, sizes in enumerate(INT8_GEMV.values()):
        got = choose("int8", [(M, N, K) for M, N in sizes for K in GEMV_DEPTHS])
        assert {g[0] for g in got} == {len(INT8_TILES) + i}
        assert {M for M, _ in sizes} == {1, 2, 3, 4}
