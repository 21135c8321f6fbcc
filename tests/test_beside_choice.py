"""CPU-only: what the kernels of the log probabilities and the adapters assume of
the split of their work, over the whole range of sizes; and that the sizes of
their GPU tests reach every kernel."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mxfp4_weight_streaming_amd", "csrc")

ROWS = [1, 2, 3, 4, 7, 16, 60, 127, 128, 129, 200, 255, 256, 257, 511, 512, 513, 1000, 1024, 1025, 2048, 5000, 1 << 20,
        2 ** 31 - 1]
VOCABS = [1, 2, 1023, 1024, 1025, 4095, 4096, 4097, 8192, 8193, 16383, 16384, 16385, 20000, 32771, 65536, 65537, 157184, 262144,
          262145, 1000003, 1 << 24, 1 << 30]


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    exe = tmp_path_factory.mktemp("choice") / "beside_choice"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "beside_choice.cpp")], check=True)

    def run(op, sizes):
        text = "".join(f"{op} {' '.join(map(str, s))}\n" for s in sizes)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(list(sizes))
        return got

    return run


def test_logprob_plans(choose):
    sizes = [(M, V) for M in ROWS for V in VOCABS]
    for (M, V), (threads, segments, each, groups, parts, part) in zip(sizes, choose("logprobs", sizes)):
        if threads == 64:                                # a wave holds the row
            assert V <= 6144 and parts == 1 and segments == -(-V // 1024)
            continue
        assert threads in (256, 512, 1024) and V > 2048
        assert (segments - 1) * 16 * threads < V <= segments * 16 * threads
        assert (groups - 1) * each < segments <= groups * each
        assert (segments + threads * 16) * threads * 16 < 2 ** 63
        if parts == 1:
            assert groups <= 16                          # a thread's registers, and 64 KB of LDS at 1,024 threads
        else:
            assert threads == 256 and groups <= 64 and 2 <= parts <= 64   # a lane a part
            assert part % each == 0                      # whole groups
            assert (parts - 1) * part < segments <= parts * part


def test_logprob_tests_reach_every_kernel(choose):
    """Sizes of tests/test_gpu_logprobs.py."""
    sizes = [(5, 8191), (300, 5003), (1025, 1000), (17, 2048), (512, 4096), (1024, 6144), (1, 157184), (64, 40000),
             (130, 262144), (130, 300007), (300, 30011), (600, 20011), (128, 16400), (129, 16400), (1, 1000003)]
    got = choose("logprobs", sizes)
    kinds = {(g[0], g[4] > 1) for g in got}
    assert kinds == {(64, False), (256, False), (512, False), (1024, False), (256, True)}
    assert {g[1] for g in got if g[0] == 64} == {1, 2, 4, 6}
    assert any(g[2] > 1 and g[4] > 1 for g in got) and any(g[2] > 1 and g[4] == 1 for g in got)   # groups of several segments


def test_adapter_plans(choose):
    sizes = [(M, N, K, r) for M in ROWS for N in (1, 16, 255, 257, 2560, 157184, 2 ** 31 - 1) for K in (1, 8, 2560, 8192)
             for r in (1, 8, 16, 17, 32, 33, 64, 128)]
    for (M, N, K, r), (few, fused, shrink, expand, rows) in zip(sizes, choose("lora", sizes)):
        assert shrink in (1, 2, 4, 8, 16) and expand in (1, 2, 4, 8, 16)
        assert not fused or (few and K >= 8 and r <= 16)
        assert few == (M * (-(-r // 32) * 32) <= 16384 and M * r * (K + N) <= 48 << 20)
        assert rows >= 256 and rows % 256 == 0 and (rows == 256 or rows * N <= 1 << 26)


def test_adapter_tests_reach_every_kernel(choose):
    """The sizes of tests/test_gpu_lora.py: fused and not, few and many, with slots and without."""
    got = choose("lora", [(1, 2560, 2560, 16), (70, 65, 257, 33), (9, 200, 96, 16), (1, 70, 130, 16), (300, 48, 64, 128),
                          (512, 1024, 2560, 64), (2048, 768, 512, 16), (130, 2563, 769, 100),
                          (16, 60000, 256, 64), (60, 3400, 3300, 128)])
    assert [g[0] for g in got[-2:]] == [0, 0]            # few tokens that would read too much by themselves
    assert {(g[0], g[1]) for g in got} == {(1, 1), (1, 0), (0, 0)}
    many = [g for g in got if not g[0]]
    assert any(g[2] > 1 for g in many) and any(g[3] > 1 for g in many)
