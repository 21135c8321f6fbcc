"""CPU-only: the sizes of the GPU tests in tests/_beside_sizes.py reach every
kernel and every way of splitting a row, by the library's own rules."""
from _beside_sizes import LOGPROB_ROWS, LOGPROB_SHORT_ROWS
from test_beside_choice import choose  # noqa: F401


def test_rows_of_every_kind_reach_every_split(choose):  # noqa: F811
    plans = {(threads, segments > 1, each > 1, parts > 1)
             for threads, segments, each, groups, parts, part in choose("logprobs", LOGPROB_ROWS)}
    assert plans == {(256, True, False, False), (256, True, True, False), (512, True, False, False), (512, True, True, False),
                     (1024, True, False, False), (1024, True, True, False), (512, False, False, False), (1024, False, False, False),
                     (256, True, False, True), (256, True, True, True)}
    short = choose("logprobs", LOGPROB_SHORT_ROWS)
    assert {p[0] for p in short} == {64} and {p[1] for p in short} == {1, 2, 4, 5, 6}


def test_one_launch_for_few_tokens(choose):  # noqa: F811
    """By what it costs: workgroups a compute unit, the steps along K of each (twice where K is odd), and the rank."""
    def fused(rank, K, N=2560):
        """The largest number of workgroups a compute unit (of 256), in quarters, that are one launch."""
        tiles = -(-N // 256)
        got = choose("lora", [(max(1, 64 * q // tiles), N, K, rank) for q in range(1, 17)])
        one = [g[1] for g in got]
        assert one == sorted(one, reverse=True)          # from some number on it is two
        return sum(one) / 4

    for N in (512, 2560, 20000):
        assert [fused(16, K, N) for K in (8, 64, 1026, 2048, 2558, 2560)] == [3.0] * 6
        assert [fused(8, K, N) for K in (8, 2560)] == [3.0] * 2
        assert [fused(13, K, N) for K in (9, 769, 2559, 2562, 4096, 5120)] == [2.0] * 6
        assert [fused(16, K, N) for K in (2561, 5119, 5122, 7680, 8192, 8193, 16384)] == [1.0] * 7
        assert [fused(5, K, N) for K in (9, 769, 4096, 4095, 8192)] == [1.0] * 5
        assert [fused(8, K, N) for K in (7, 5121, 10242)] == [fused(16, K, N) for K in (7, 10241, 20482)] == [0.0] * 3
    assert fused(17, 64) == 0.0
