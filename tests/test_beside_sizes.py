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
