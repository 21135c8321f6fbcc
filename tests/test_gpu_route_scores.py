"""moe_route_scores against a plain implementation in 64 bits that sorts.

ids are compared for equality (the scores are fp64 evaluations rounded to fp32
on both sides).  A weight is s / sum * factor of these fp32 scores, with K - 1
additions, a division and a product in fp32, and the two sides' scores may be
one rounding (2^-24) apart: relative error at most (1 + (1 + K - 1) + 1 + 1)
2^-24 with K = 8, that is 11 * 2^-24 < 6.6e-7, plus the smallest fp32 numbers for
weights that underflow.
"""
import numpy as np
import pytest
import torch

from _around_gpu import Out, up
from _around_ref import route

pytestmark = pytest.mark.gpu

NEG = -np.inf


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _check(moe, logits, bias, K, **kw):
    M, E = logits.shape
    ids, w = Out((M, K), torch.int32), Out((M, K), torch.float32)
    moe.moe_route_scores(moe.router(E, K, **kw), up(logits), None if bias is None else up(bias), ids.t, w.t)
    torch.cuda.synchronize()
    ri, rw = route(logits, bias, K, **kw)
    gi, gw = ids.bits(), w.bits()
    bad = np.nonzero((gi != ri).any(1))[0]
    assert bad.size == 0, (bad[:3], gi[bad[:3]], ri[bad[:3]])
    assert np.all(np.abs(gw - rw) <= 6.6e-7 * np.abs(rw) + 1e-44), np.max(np.abs(gw - rw) / (np.abs(rw) + 1e-300))
    return gi, gw


# experts, K, groups, groups kept: one expert, below and around a wave, odd sizes, groups of one, every group kept
CASES = [(1, 1, 1, 1), (2, 2, 1, 1), (8, 8, 1, 1), (16, 2, 1, 1), (60, 4, 4, 2), (63, 7, 9, 5), (64, 8, 64, 8),
         (64, 6, 8, 3), (65, 5, 5, 2), (96, 3, 16, 15), (100, 1, 4, 4), (128, 8, 8, 4), (160, 6, 8, 3), (255, 8, 5, 1),
         (256, 8, 1, 1), (256, 8, 8, 4), (257, 8, 1, 1), (320, 7, 16, 14), (384, 8, 2, 1), (511, 8, 7, 3),
         (129, 6, 43, 20), (495, 8, 55, 7), (512, 8, 1, 1), (512, 8, 8, 4), (512, 8, 64, 1), (512, 8, 16, 8)]


@pytest.mark.parametrize("E,K,G,keep", CASES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_sizes(moe, E, K, G, keep, score):
    rng = np.random.default_rng(100 * E + K)
    for M, with_bias, n, renorm in ((1, True, 2, True), (6, False, 2, True), (70, True, 1, False)):
        logits = rng.standard_normal((M, E)).astype(np.float32)
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
        _check(moe, logits, bias, K, score=score, groups=G, group_topk=keep, group_score=n, renormalise=renorm,
               factor=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(512, 8, 4), (256, 1, 1), (60, 6, 3)])
def test_many_tokens(moe, score, E, G, keep):
    rng = np.random.default_rng(9)
    logits = (rng.standard_normal((1500, E)) * np.exp(rng.standard_normal((1500, 1)))).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    _check(moe, logits, bias, 8, score=score, groups=G, group_topk=keep)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(256, 8, 4), (512, 1, 1), (45, 5, 2)])
def test_ties(moe, score, E, G, keep):
    """Whole rows of equal logits, and few distinct values: the lowest index of groups and of experts wins."""
    rng = np.random.default_rng(10)
    logits = rng.integers(-2, 3, (40, E)).astype(np.float32)
    logits[0] = 0.0
    logits[1] = -0.0
    logits[2, ::2] = 0.0
    logits[2, 1::2] = -0.0
    for bias in (None, np.zeros(E, np.float32), (0.5 * rng.integers(-1, 2, E)).astype(np.float32)):
        for n in (1, 2):
            _check(moe, logits, bias, 8, score=score, groups=G, group_topk=keep, group_score=n)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(256, 8, 4), (512, 16, 2), (64, 1, 1), (63, 7, 2)])
def test_unavailable_experts(moe, score, E, G, keep):
    """-inf and NaN logits and biases, the lowest finite value, rows and groups with nothing left."""
    rng = np.random.default_rng(11)
    logits = rng.standard_normal((30, E)).astype(np.float32)
    logits[rng.random((30, E)) < 0.5] = NEG
    logits[0] = NEG                                       # nothing left
    logits[1] = np.nan
    logits[2] = NEG
    logits[2, E // 2] = 0.3                               # one left
    logits[3] = np.finfo(np.float32).min                  # available, score 0
    logits[4, : E // 2] = NEG
    logits[5, ::3] = np.nan
    logits[6, 5] = np.inf                                 # counts as the largest finite value
    logits[7, 3:9] = np.inf
    logits[8] = np.finfo(np.float32).max
    logits[9] = -200.0                                    # sigmoid underflows in fp32
    logits[10] = 100.0                                    # sigmoid is 1
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias_gone = bias.copy()
    bias_gone[:: 4] = NEG
    bias_gone[1] = np.nan
    for b in (None, bias, bias_gone, bias - np.float32(3.0)):
        gi, gw = _check(moe, logits, b, 8, score=score, groups=G, group_topk=keep, factor=1.5)
        assert not gw[0].any() and not gw[1].any()
        assert all(len(set(r)) == 8 for r in gi.tolist())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("forced", [3, 8, 40, 200])
@pytest.mark.parametrize("G,keep", [(1, 1), (8, 4)])
def test_forced_and_large_biases(moe, score, forced, G, keep):
    """+inf biases force experts (the lowest indexes first where they are many); huge ones swallow the scores."""
    rng = np.random.default_rng(14)
    logits = rng.standard_normal((20, 256)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(256)).astype(np.float32)
    at = rng.permutation(256)[:forced]
    for v in (np.inf, 1e30, -1e30, 3e7):
        b = bias.copy()
        b[at] = v
        _check(moe, logits, b, 8, score=score, groups=G, group_topk=keep)


@pytest.mark.parametrize("size", [1.0, 30.0, 1000.0, 3e5])
@pytest.mark.parametrize("E,G,keep", [(256, 8, 4), (512, 64, 9), (48, 24, 7)])
def test_groups_of_opposite_biases(moe, size, E, G, keep):
    """Two available experts a group whose large biases cancel in the group's value, to the last bits."""
    rng = np.random.default_rng(15)
    logits = np.full((200, E), NEG, np.float32)
    bias = np.zeros(E, np.float32)
    for g in range(G):
        a, b = g * (E // G), g * (E // G) + 1
        logits[:, [a, b]] = rng.standard_normal((200, 2)).astype(np.float32)
        bias[a], bias[b] = size, -size
    _check(moe, logits, bias, 4, score="sigmoid", groups=G, group_topk=keep)


def test_near_values(moe):
    """Scores that are neighbours in fp32: the order of the correctly rounded scores decides."""
    rng = np.random.default_rng(12)
    base = rng.standard_normal((200, 1)).astype(np.float32)
    steps = rng.integers(-6, 7, (200, 128)).astype(np.int32)
    logits = (np.ascontiguousarray(np.broadcast_to(base, (200, 128))).view(np.int32) + steps).view(np.float32)
    for score in ("sigmoid", "softmax"):
        _check(moe, logits, None, 8, score=score)
        _check(moe, logits, np.full(128, 0.25, np.float32), 8, score=score, groups=8, group_topk=2)


def test_weights_of_one_selected(moe):
    logits = np.array([[0.0, 3.0, -1.0]], np.float32)
    gi, gw = _check(moe, logits, None, 1, score="sigmoid", factor=2.0)
    assert gi.tolist() == [[1]] and gw.tolist() == [[2.0]]


@pytest.mark.parametrize("M,H,I,E,K", [(1, 2560, 768, 256, 8), (8, 256, 64, 16, 2), (40, 2560, 768, 64, 8)])
def test_router_logits_are_the_layers(moe, M, H, I, E, K):
    from mxfp4_weight_streaming_amd import synth
    rng = np.random.default_rng(13)
    x, wr = synth.normal_bf16(rng, (M, H), 1.0), synth.normal_bf16(rng, (E, H), 0.02)
    shp = moe.shape(H, I, E, K)
    got, tap = Out((M, E), torch.float32), Out((M, E), torch.float32)
    moe.moe_router_logits(shp, M, up(x), up(wr), got.t)
    ws = moe.workspace(shp, M)
    ids, w = Out((M, K), torch.int32), Out((M, K), torch.float32)
    moe.moe_route(shp, M, up(x), up(wr), ids.t, w.t, ws, taps={"logits": tap.t})
    torch.cuda.synchronize()
    assert np.array_equal(got.bits().view(np.uint32), tap.bits().view(np.uint32))
    ref = synth.bf16_to_f32(x).astype(np.float64) @ synth.bf16_to_f32(wr).astype(np.float64).T
    mag = np.abs(synth.bf16_to_f32(x)).astype(np.float64) @ np.abs(synth.bf16_to_f32(wr)).astype(np.float64).T
    assert np.all(np.abs(got.bits() - ref) <= H * 2.0 ** -24 * mag)      # H fp32 additions of exact products
