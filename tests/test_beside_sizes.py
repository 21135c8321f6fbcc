"""CPU-only: the sizes of the GPU tests in tests/_beside_sizes.py reach every
kernel and every way of splitting a row, by the library's own rules."""
from _beside_sizes import LOGPROB_ROWS, LOGPROB_SHORT_ROWS, LORA_CHANNELS, LORA_DEPTHS, LORA_LARGE, LORA_RANKS
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


def test_adapters_of_many_tokens_reach_every_form(choose):  # noqa: F811
    """All on the matrix cores; one and two tiles of ranks a workgroup, steps of 32 ranks, rows of B of less than 8 and of
    no multiple of 8, depths below a load, below a step and between."""
    sizes = LORA_RANKS + LORA_DEPTHS + LORA_CHANNELS + LORA_LARGE
    got = choose("lora", [(M, N, K, r) for M, r, K, N in sizes])
    assert all(g[0] == 0 for g in got)
    # (two tiles, steps, less than 8, ending inside 8)
    forms = lambda which: {(r > 16, 1 if r <= 32 else 2 if r <= 64 else 4, r < 8, r > 8 and r % 8 != 0) for _, r, _, _ in which}  # noqa: E731
    every = {(False, 1, True, False), (False, 1, False, False), (False, 1, False, True), (True, 1, False, False), (True, 1, False, True),
             (True, 2, False, False), (True, 2, False, True), (True, 4, False, False), (True, 4, False, True)}
    assert forms(LORA_RANKS) == every
    assert any(65 <= r <= 96 for _, r, _, _ in LORA_RANKS)   # four steps' kernel with three
    for r in (13, 16, 40):
        depths = {K for _, rank, K, _ in LORA_DEPTHS if rank == r}
        assert {1, 7, 8, 9, 63, 64, 65} <= depths and any(K > 2560 for K in depths)
    assert {N % 4 for _, _, _, N in LORA_CHANNELS} == {0, 1, 2, 3} and min(N for _, _, _, N in LORA_CHANNELS) == 1
    assert {1} < {g[2] for g in got} and {1} < {g[3] for g in got}
    large = choose("lora", [(M, N, K, r) for M, r, K, N in LORA_LARGE])
    assert any(g[2] == 1 for g in large) and any(g[3] == 1 for g in large)
