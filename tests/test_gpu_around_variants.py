"""Every kernel variant of the operators around the expert layer, by sizes that
choose it (tests/_around_variants.py), bit for bit: the int8 product against
exact sums, the norm and the quantiser against their plain forms; routing of
more tokens than the chip holds waves, token for token against the plain
implementation; the largest tile in a graph; more rows than a launch has
workgroups, and tensors beyond 2^31 elements.
"""
import numpy as np
import pytest
import torch

import oracle
from _around_gpu import Out, same_f32, up
from _around_ref import int8_rows, rmsnorm, route
from _around_variants import GEMV_DEPTHS, INT8_GEMV, INT8_TILES, NORM, QUANT, tile_depths
from mxfp4_weight_streaming_amd import synth

pytestmark = pytest.mark.gpu

BF, F32, I8, F8 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


# ---- int8 product ---------------------------------------------------------------
def _product(M, N, K, seed):
    """Inputs, and the definition's outputs in both types: sums of integers below 2^53 are exact in fp64."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=I8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=I8)
    sa = 0.01 + torch.rand(M, generator=g, device="cuda")
    sw = 0.001 + 0.01 * torch.rand(N, generator=g, device="cuda")
    acc = a.double() @ w.double().t()
    ref = (acc.float() * sa[:, None]) * sw[None, :]
    return (a, sa, w, sw), {F32: ref, BF: ref.to(BF)}


def _run_product(moe, M, N, K, types):
    args, ref = _product(M, N, K, M + 3 * N + 7 * K)
    for t in types:
        out = Out((M, N), t)
        moe.moe_int8_linear(*args, out.t)
        torch.cuda.synchronize()
        assert bool((out.raw[out.n:] == 0xA5).all()), "written behind the output"
        bits = torch.int32 if t == F32 else torch.int16
        off = torch.nonzero(out.t.view(bits) != ref[t].view(bits))
        assert off.numel() == 0, (off.shape[0], off[:4].tolist())


@pytest.mark.parametrize("M,N,step,ring", [pytest.param(M, N, *step_ring, id=f"{tile}-{M}x{N}")
                                           for tile, (step_ring, sizes) in INT8_TILES.items() for M, N in sizes])
def test_int8_tiles(moe, M, N, step, ring):
    for i, K in enumerate(tile_depths(step, ring)):
        print(f"{M} x {N} x {K}", flush=True)
        _run_product(moe, M, N, K, (F32, BF) if i % 4 == 0 else ((F32,) if i % 2 else (BF,)))


@pytest.mark.parametrize("M,N", [pytest.param(M, N, id=f"{v}-{M}x{N}") for v, sizes in INT8_GEMV.items() for M, N in sizes])
def test_int8_gemv(moe, M, N):
    for K in GEMV_DEPTHS:
        print(f"{M} x {N} x {K}", flush=True)
        _run_product(moe, M, N, K, (F32, BF))


@pytest.mark.parametrize("M,N,K", [(768, 20480, 832), (129, 20003, 640), (300, 5121, 641)])
def test_int8_tiles_in_a_graph(moe, M, N, K):
    """Tiles of more than 64 KB of LDS and others, captured, replayed between eager calls."""
    args, ref = _product(M, N, K, 5)
    out, other = Out((M, N), BF), Out((M, N), F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        moe.moe_int8_linear(*args, out.t)
    for _ in range(4):
        out.t.zero_()
        g.replay()
        moe.moe_int8_linear(*args, other.t)
        torch.cuda.synchronize()
        assert torch.equal(out.t.view(torch.int16), ref[BF].view(torch.int16))
        assert torch.equal(other.t.view(torch.int32), ref[F32].view(torch.int32))


# ---- norm and quantiser -----------------------------------------------------------
@pytest.mark.parametrize("M,H", NORM)
def test_norm(moe, M, H):
    rng = np.random.default_rng(M + 5 * H)
    for xb, rb, q in ((False, True, F8), (True, False, I8), (False, False, None), (True, True, F8)):
        x, res = rng.standard_normal((2, M, H)).astype(np.float32) * [[[1.0]], [[2.0]]]
        x, res = x.astype(np.float32), res.astype(np.float32)
        x = synth.bf16_from_f32(x) if xb else x
        res = synth.bf16_from_f32(res) if rb else res
        w = synth.bf16_from_f32((1 + 0.2 * rng.standard_normal(H)).astype(np.float32))
        r, yb, _ = rmsnorm(x, res, w, 1e-6, rb)
        ro, y = Out((M, H), BF if rb else F32), Out((M, H), BF)
        codes, scale = (None, None) if q is None else (Out((M, H), q), Out((M,), F32))
        print(f"{M} x {H} {xb} {rb} {q}", flush=True)
        moe.moe_add_rmsnorm(up(x), up(res), up(w), 1e-6, ro.t, y=y.t, q=None if q is None else codes.t,
                            scale=None if q is None else scale.t)
        torch.cuda.synchronize()
        assert np.array_equal(ro.bits().view(np.uint8), r.view(np.uint8))
        assert np.array_equal(y.bits(), yb)
        if q is not None:
            rq, rs = oracle.quant_act(yb) if q == F8 else int8_rows(yb)
            assert same_f32(scale.bits(), rs) and np.array_equal(codes.bits().view(np.uint8), rq.view(np.uint8))


@pytest.mark.parametrize("rows,cols", QUANT)
def test_quantise(moe, rows, cols):
    rng = np.random.default_rng(rows + 3 * cols)
    v = synth.bf16_from_f32((rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32))
    v[rows // 2] = 0
    q, s = Out((rows, cols), I8), Out((rows,), F32)
    moe.moe_int8_quantize(up(v), q.t, s.t)
    torch.cuda.synchronize()
    rq, rs = int8_rows(v)
    assert same_f32(s.bits(), rs) and np.array_equal(q.bits(), rq)


# ---- routing ----------------------------------------------------------------------
def _tokens(rng, E, each):
    """Tokens that take each way through the kernel: plain, equal logits, few values, groups within the fp32 scores'
    error of each other, little or nothing available, forced beyond the scores' range."""
    plain = rng.standard_normal((60, E)).astype(np.float32)
    equal = np.zeros((20, E), np.float32)
    few = rng.integers(-2, 3, (40, E)).astype(np.float32)
    group = np.tile(rng.standard_normal((20, each)).astype(np.float32), (1, -(-E // each)))[:, :E].copy()
    gone = rng.standard_normal((40, E)).astype(np.float32)
    gone[rng.random((40, E)) < 0.9] = -np.inf
    none = np.full((20, E), -np.inf, np.float32)
    none[::2] = np.nan
    far = (rng.standard_normal((20, E)) * 300).astype(np.float32)
    return np.concatenate([plain, equal, few, group, gone, none, far])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(512, 8, 4), (256, 1, 1), (160, 8, 3), (510, 2, 1), (60, 6, 3)])
def test_routing_of_more_tokens_than_waves(moe, score, E, G, keep):
    """A wave takes several tokens, one after another through the same LDS: each as if it were alone."""
    rng = np.random.default_rng(17)
    K, M = 8, 20011
    kinds = _tokens(rng, E, E // G)
    for bias, n in ((None, 2), ((0.05 * rng.standard_normal(E)).astype(np.float32), 1)):
        opts = dict(score=score, groups=G, group_topk=keep, group_score=n, factor=1.5)
        ri, rw = route(kinds, bias, K, **opts)
        at = rng.integers(0, len(kinds), M)
        ids, w = Out((M, K), torch.int32), Out((M, K), F32)
        moe.moe_route_scores(moe.router(E, K, **opts), up(kinds[at]), None if bias is None else up(bias), ids.t, w.t)
        torch.cuda.synchronize()
        bad = np.nonzero((ids.bits() != ri[at]).any(1))[0]
        assert bad.size == 0, (bad[:3], at[bad[:3]])
        gw = w.bits()
        # a weight is a quotient of fp32 scores and their sum, times the factor: 11 roundings at most
        assert np.all(np.abs(gw - rw[at]) <= 6.6e-7 * np.abs(rw[at]) + 1e-44)
        # the same token has the same bits wherever it stands
        first = np.zeros(len(kinds), np.int64)
        first[at[::-1]] = np.arange(M)[::-1]
        assert same_f32(gw, gw[first[at]])


# ---- many rows: workgroups that take a second row, offsets beyond 32 bits ---------------
def _repeats(t, ref):
    """Whether the rows of t are those of ref over and over, bit for bit."""
    n = ref.shape[0]
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    t, ref = t.view(bits), ref.view(bits)
    whole = t.shape[0] // n * n
    return bool((t[:whole].unflatten(0, (-1, n)) == ref).all()) and torch.equal(t[whole:], ref[: t.shape[0] - whole])


@pytest.mark.parametrize("M,H,kept", [((1 << 20) + 1003, 2051, 512), ((1 << 20) + 1003, 1025, 256), ((1 << 24) + 77, 129, 16)])
def test_norm_of_more_rows_than_workgroups(moe, M, H, kept):
    """Rows that repeat give the bits of one set of them, wherever they stand."""
    rng = np.random.default_rng(H)
    x = synth.bf16_from_f32((rng.standard_normal((kept, H)) * np.exp(rng.standard_normal((kept, 1)))).astype(np.float32))
    w = synth.bf16_from_f32((1 + 0.2 * rng.standard_normal(H)).astype(np.float32))
    _, yb, _ = rmsnorm(x, None, w, 1e-6, True)
    rq, rs = int8_rows(yb)
    dx = up(x).repeat(-(-M // kept), 1)[:M].contiguous()
    y, q, s = Out((M, H), BF), Out((M, H), I8), Out((M,), F32)
    moe.moe_add_rmsnorm(dx, None, up(w), 1e-6, None, y=y.t, q=q.t, scale=s.t)
    torch.cuda.synchronize()
    for o, ref in ((y, up(yb)), (q, up(rq)), (s, up(rs))):
        assert bool((o.raw[o.n:] == 0xA5).all()) and _repeats(o.t, ref)
    # and the quantiser alone, on the norm's rows
    q.t.zero_(), s.t.zero_()
    moe.moe_int8_quantize(y.t, q.t, s.t)
    torch.cuda.synchronize()
    for o, ref in ((q, up(rq)), (s, up(rs))):
        assert bool((o.raw[o.n:] == 0xA5).all()) and _repeats(o.t, ref)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_routing_offsets_beyond_32_bits(moe, score):
    rng = np.random.default_rng(18)
    E, K, M, kept = 512, 8, (1 << 22) + 300_001, 400
    logits = rng.standard_normal((kept, E)).astype(np.float32)
    opts = dict(score=score, groups=8, group_topk=4, factor=2.5)
    ri, rw = route(logits, None, K, **opts)
    dl = up(logits).repeat(-(-M // kept), 1)[:M].contiguous()
    ids, w = Out((M, K), torch.int32), Out((M, K), F32)
    moe.moe_route_scores(moe.router(E, K, **opts), dl, None, ids.t, w.t)
    torch.cuda.synchronize()
    assert bool((ids.raw[ids.n:] == 0xA5).all()) and bool((w.raw[w.n:] == 0xA5).all())
    assert _repeats(ids.t, up(ri)) and _repeats(w.t, w.t[:kept].clone())
    assert np.all(np.abs(w.t[:kept].cpu().numpy() - rw) <= 6.6e-7 * np.abs(rw) + 1e-44)


@pytest.mark.parametrize("M,N,K", [(70001, 40, 65536), (70001, 40, 65537), (1, 70001, 65536), (3, 70001, 65537),
                                   (9, 70001, 65552)])
def test_int8_inputs_beyond_32_bits(moe, M, N, K):
    """Codes of more than 2^32 bytes: sampled rows, the first and last among them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(19)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=I8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=I8)
    sa, sw = 0.5 + torch.rand(M, generator=g, device="cuda"), 0.5 + torch.rand(N, generator=g, device="cuda")
    out = Out((M, N), F32)
    moe.moe_int8_linear(a, sa, w, sw, out.t)
    torch.cuda.synchronize()
    assert bool((out.raw[out.n:] == 0xA5).all())
    for m in {0, M // 2, max(0, M - 300)}:
        for n in {0, N // 2, max(0, N - 300)}:
            rows, cols = slice(m, m + 300), slice(n, n + 300)
            ref = ((a[rows].double() @ w[cols].double().t()).float() * sa[rows, None]) * sw[None, cols]
            assert torch.equal(out.t[rows, cols].contiguous().view(torch.int32), ref.view(torch.int32))
