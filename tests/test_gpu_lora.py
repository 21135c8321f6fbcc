"""moe_lora_add and moe_int8_linear_lora against sums in 64 bits
(tests/_beside_ref.py)."""
import numpy as np
import pytest
import torch

from _around_gpu import Out
from _beside_ref import check_rows, lora_delta

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _adapters(g, L, r, K, N, scale=True):
    a = (torch.randn(L, r, K, generator=g) / K ** 0.5).to(torch.bfloat16)
    b = (torch.randn(L, N, r, generator=g) / r ** 0.5).to(torch.bfloat16)
    return a, b, 0.5 + torch.rand(L, generator=g) if scale else None


def _ids(g, M, L, kind):
    """Requests' tokens one after another, or tokens in any order; some without an adapter, some with ids outside."""
    if kind == "runs":
        ids = torch.randint(-1, L, (M // 7 + 1,), generator=g).repeat_interleave(7)[:M]
    elif kind == "one":
        ids = torch.full((M,), L - 1)
    else:
        ids = torch.randint(-1, L, (M,), generator=g)
        ids[torch.rand(M, generator=g) < 0.05] = L
        ids[torch.rand(M, generator=g) < 0.05] = -2 ** 31
    return ids.to(torch.int32)


def _add(moe, a, b, scale, x, ids, base, dtype, in_place=False):
    lp = moe.lora(a.cuda(), b.cuda(), None if scale is None else scale.cuda())
    M, N = x.shape[0], b.shape[1]
    ws = moe.lora_workspace(lp, M)
    ws.fill_(0xFF)
    out = Out((M, N), dtype)
    src = None if base is None else base.cuda()
    if in_place:
        out.t.copy_(src)
        src = out.t
    moe.moe_lora_add(lp, x.cuda(), ids.cuda(), src, out.t, ws)
    torch.cuda.synchronize()
    out.bits()                                           # (checks what is behind it)
    return out.t


def _check_add(moe, seed, M, L, r, K, N, dtype, kind="any", base=True, scale=True, in_place=False):
    print(f"M={M} L={L} r={r} K={K} N={N} {dtype} {kind}", flush=True)
    g = torch.Generator().manual_seed(seed)
    a, b, s = _adapters(g, L, r, K, N, scale)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    y = torch.randn(M, N, generator=g).to(dtype) if base else None
    ids = _ids(g, M, L, kind)
    got = _add(moe, a, b, s, x, ids, y, dtype, in_place)
    d, err = lora_delta(x, a, b, s, ids)
    check_rows(got, d + (0 if y is None else y.double()), err, dtype)
    if y is not None:
        bare = (ids < 0) | (ids >= L)
        assert torch.equal(got.cpu()[bare], y[bare])     # a token without an adapter keeps its row


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 33, 64, 65, 129, 257])
def test_tokens(moe, M, dtype):
    for n, (L, r, K, N) in enumerate(((3, 16, 256, 320), (1, 8, 64, 64), (20, 13, 77, 131), (5, 64, 520, 96))):
        _check_add(moe, M + n, M, L, r, K, N, dtype, ("any", "one", "runs", "any")[n])


@pytest.mark.parametrize("r", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 40, 48, 63, 64, 65, 96, 127, 128])
def test_ranks(moe, r):
    for M, K, N in ((1, 130, 70), (9, 96, 200), (70, 257, 65), (300, 64, 48)):
        _check_add(moe, r + M, M, 4, r, K, N, torch.float32)


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 31, 32, 33, 63, 65, 127, 511, 513, 1000, 2560, 2561])
def test_depths(moe, K):
    for M in (1, 6, 40, 200):
        _check_add(moe, K + M, M, 3, 16, K, 80, torch.float32, "runs")


@pytest.mark.parametrize("N", [1, 2, 3, 5, 8, 15, 17, 63, 65, 255, 257, 1001, 4099])
def test_channels(moe, N):
    for M, dtype in ((1, torch.bfloat16), (6, torch.float32), (40, torch.bfloat16), (200, torch.float32)):
        for r in (8, 11):
            _check_add(moe, N + M, M, 3, r, 48, N, dtype)


@pytest.mark.parametrize("M,L,r,K,N,dtype,kind", [
    (1, 8, 16, 2560, 2560, torch.bfloat16, "one"), (64, 64, 16, 2560, 2560, torch.bfloat16, "any"),
    (4, 8, 16, 2560, 20000, torch.float32, "any"), (512, 8, 64, 2560, 1024, torch.bfloat16, "runs"),
    (2048, 6, 16, 512, 768, torch.bfloat16, "runs"), (1000, 40, 32, 300, 300, torch.float32, "any"),
    (8, 300, 128, 4096, 64, torch.float32, "any"), (130, 2, 100, 769, 2563, torch.bfloat16, "runs")])
def test_shapes(moe, M, L, r, K, N, dtype, kind):
    _check_add(moe, M + r, M, L, r, K, N, dtype, kind)


@pytest.mark.parametrize("M", [1, 5, 60, 300])
def test_forms(moe, M):
    """Without a base, without scales, in place."""
    for dtype in (torch.float32, torch.bfloat16):
        _check_add(moe, M, M, 4, 16, 128, 200, dtype, base=False)
        _check_add(moe, M, M, 4, 16, 128, 200, dtype, scale=False)
        _check_add(moe, M, M, 4, 12, 130, 201, dtype, in_place=True)


@pytest.mark.parametrize("M", [2, 16, 70, 300])
@pytest.mark.parametrize("r", [5, 16, 64])
def test_rows_keep_to_their_adapter(moe, M, r):
    """Infinities and NaN in an adapter, or in a token, reach their own rows only."""
    g = torch.Generator().manual_seed(M + r)
    L, K, N = 5, 96, 130
    a, b, s = _adapters(g, L, r, K, N)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    y = torch.randn(M, N, generator=g)
    ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
    ids[0], ids[1] = 0, 1
    ref = _add(moe, a, b, s, x, ids, y, torch.float32)
    a2, b2, x2 = a.clone(), b.clone(), x.clone()
    a2[0], b2[2], x2[1] = float("nan"), float("inf"), float("inf")
    s2 = s.clone()
    s2[3] = float("nan")
    got = _add(moe, a2, b2, s2, x2, ids, y, torch.float32)
    same = (ids != 0) & (ids != 2) & (ids != 3)
    same[1] = False
    assert torch.equal(got[same.cuda()], ref[same.cuda()])
    assert not bool(torch.isfinite(got[0]).any())


def test_repeated_call_is_the_same(moe):
    g = torch.Generator().manual_seed(4)
    a, b, s = _adapters(g, 6, 16, 512, 640)
    for M in (1, 40, 600):
        x = torch.randn(M, 512, generator=g).to(torch.bfloat16)
        ids = _ids(g, M, 6, "any")
        y = torch.randn(M, 640, generator=g)
        first = _add(moe, a, b, s, x, ids, y, torch.float32)
        for _ in range(3):
            assert torch.equal(_add(moe, a, b, s, x, ids, y, torch.float32), first)


def test_offsets_beyond_32_bits(moe):
    """Adapters whose weights stand beyond 2^31 elements."""
    L, r, K, N = 2100, 128, 8192, 40
    a = torch.zeros(L, r, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(L, N, r, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(2)
    la, lb, _ = _adapters(g, 1, r, K, N)
    a[L - 1], b[L - 1] = la[0].cuda(), lb[0].cuda()
    lp = moe.lora(a, b)
    for M in (1, 5, 200):
        x = torch.randn(M, K, generator=g).to(torch.bfloat16)
        ids = torch.full((M,), L - 1, dtype=torch.int32)
        out = Out((M, N), torch.float32)
        moe.moe_lora_add(lp, x.cuda(), ids.cuda(), None, out.t, moe.lora_workspace(lp, M))
        torch.cuda.synchronize()
        d, err = lora_delta(x, la, lb, None, torch.zeros(M, dtype=torch.int32))
        check_rows(out.bits(), d, err, torch.float32)


# ---- with the int8 projection ---------------------------------------------------
def _check_int8(moe, seed, M, L, r, K, N, dtype, kind="any"):
    print(f"M={M} L={L} r={r} K={K} N={N} {dtype} {kind}", flush=True)
    g = torch.Generator().manual_seed(seed)
    a, b, s = _adapters(g, L, r, K, N)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    q = torch.randint(-127, 128, (M, K), generator=g).to(torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8)
    qs, ws = (0.01 + torch.rand(M, generator=g)) / K ** 0.5 / 50, (0.01 + torch.rand(N, generator=g)) / 50
    ids = _ids(g, M, L, kind)
    lp = moe.lora(a.cuda(), b.cuda(), s.cuda())
    scratch = moe.lora_workspace(lp, M)
    scratch.fill_(0xFF)
    out, plain = Out((M, N), dtype), Out((M, N), dtype)
    dev = [t.cuda() for t in (q, qs, w, ws)]
    moe.moe_int8_linear_lora(*dev, lp, x.cuda(), ids.cuda(), out.t, scratch)
    moe.moe_int8_linear(*dev, plain.t)
    torch.cuda.synchronize()
    out.bits()
    base = (q.double() @ w.double().t()) * qs.double()[:, None] * ws.double()
    d, err = lora_delta(x, a, b, s, ids)
    # (the product's own two roundings, of its value and not of the sum's)
    check_rows(out.t, base + d, err + 2.0 ** -22 * base.abs(), dtype)
    bare = ((ids < 0) | (ids >= L)).cuda()
    assert torch.equal(out.t[bare], plain.t[bare])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 16, 17, 33, 64, 65, 129, 257])
def test_int8_tokens(moe, M, dtype):
    for n, (L, r, K, N) in enumerate(((3, 16, 256, 320), (20, 13, 77, 131), (5, 64, 528, 96), (2, 8, 64, 10000))):
        if M * N < 300000:
            _check_int8(moe, M + n, M, L, r, K, N, dtype, ("any", "runs", "one", "any")[n])


@pytest.mark.parametrize("M,L,r,K,N,dtype,kind", [
    (1, 8, 16, 2560, 2560, torch.bfloat16, "one"), (32, 16, 16, 2560, 2560, torch.bfloat16, "runs"),
    (77, 5, 13, 769, 2563, torch.float32, "runs"), (2048, 8, 16, 512, 1280, torch.bfloat16, "runs"),
    (600, 8, 128, 320, 1000, torch.float32, "any"), (3, 4, 16, 512, 70000, torch.float32, "any"),
    (1030, 3, 24, 1040, 520, torch.bfloat16, "runs"), (500, 40, 1, 64, 777, torch.float32, "any")])
def test_int8_shapes(moe, M, L, r, K, N, dtype, kind):
    _check_int8(moe, M + r, M, L, r, K, N, dtype, kind)


@pytest.mark.parametrize("r", [1, 3, 8, 12, 16, 20, 31, 32, 33, 64, 100, 128])
def test_int8_ranks(moe, r):
    for M, K, N in ((2, 130, 70), (9, 96, 200), (70, 257, 65), (300, 64, 300)):
        _check_int8(moe, r + M, M, 4, r, K, N, torch.float32)


def test_int8_rows_keep_to_their_adapter(moe):
    g = torch.Generator().manual_seed(8)
    for M in (3, 20, 140, 600):
        L, r, K, N = 4, 16, 96, 260
        a, b, s = _adapters(g, L, r, K, N)
        x = torch.randn(M, K, generator=g).to(torch.bfloat16)
        q = torch.randint(-127, 128, (M, K), generator=g).to(torch.int8).cuda()
        w = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda()
        qs, ws = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
        ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
        ids[0], ids[1] = 0, 1
        outs = []
        for bad in (False, True):
            if bad:
                a, b, x = a.clone(), b.clone(), x.clone()
                a[0], b[2], x[1] = float("nan"), float("-inf"), float("inf")
            lp = moe.lora(a.cuda(), b.cuda(), s.cuda())
            outs.append(torch.empty(M, N, device="cuda"))
            moe.moe_int8_linear_lora(q, qs, w, ws, lp, x.cuda(), ids.cuda(), outs[-1], moe.lora_workspace(lp, M))
        same = (ids != 0) & (ids != 2)
        same[1] = False
        assert torch.equal(outs[0][same.cuda()], outs[1][same.cuda()])
        assert not bool(torch.isfinite(outs[1][0]).any())


@pytest.mark.parametrize("M", [1, 5, 16, 70, 600])
@pytest.mark.parametrize("r", [1, 32, 64])
def test_infinite_and_largest_values(moe, M, r):
    """An activation that is infinite, and a u near fp32's largest number, give what the formula gives: all of an adapter's
    values have one sign here, so no infinity meets its opposite."""
    g = torch.Generator().manual_seed(M + r)
    L, K, N = 2, 72, 130
    pos = lambda *s: (0.5 + torch.rand(*s, generator=g)).to(torch.bfloat16)  # noqa: E731
    a, b = pos(L, r, K), pos(L, N, r) * 2.0 ** -20
    x = pos(M, K)
    ids = torch.randint(0, L, (M,), generator=g).to(torch.int32)
    x[0, 3] = torch.inf
    x[M - 1, K - 1] = torch.inf
    if M > 4:
        a[0, :, 8:] = 0.0
        a[0, :, :8] = 1.0
        x[2] = 0.0
        x[2, 0] = torch.finfo(torch.bfloat16).max
        x[2, 1] = 2.0 ** 119                             # fp32's largest but for its last bits: bf16 would round it up
        ids[2] = 0
        ids[0] = ids[M - 1] = 1                          # (0 times infinity is NaN)
    out = _add(moe, a, b, None, x, ids, None, torch.float32)
    ref, err = lora_delta(x, a, b, None, ids)
    inf = torch.isinf(ref)
    got = out.cpu().double()
    assert bool(inf[0].all()) and bool((got[inf] == torch.inf).all())
    check_rows(torch.where(inf, 0.0, got), torch.where(inf, 0.0, ref), torch.where(inf, 0.0, err), torch.float32)


@pytest.mark.parametrize("M,L,r,K,N,dtype,kind", [
    (9, 9, 40, 300, 9000, torch.float32, "any"), (7, 3, 64, 72, 20001, torch.bfloat16, "runs"), (2, 2, 9, 40, 140000, torch.bfloat16, "any"),
    (16, 16, 64, 256, 60000, torch.float32, "any"), (5, 2, 128, 130, 90001, torch.bfloat16, "any"), (3, 3, 121, 64, 160003, torch.float32, "any"),
    (60, 60, 128, 3300, 3400, torch.bfloat16, "any")])
def test_few_tokens_of_many_channels(moe, M, L, r, K, N, dtype, kind):
    """By themselves with the workgroups of the same channels side by side, and on the matrix cores where they would read
    too much."""
    _check_add(moe, M + r, M, L, r, K, N, dtype, kind)


@pytest.mark.parametrize("M", [3, 40])
def test_adapters_beyond_32_bits(moe, M):
    """The last of many adapters, beyond 2^31 values of B (and, of A, of a second set)."""
    g = torch.Generator().manual_seed(M)
    for L, r, K, N in ((220, 64, 24, 160000), (70, 128, 262144, 40)):
        a = torch.empty(L, r, K, dtype=torch.bfloat16, device="cuda")
        b = torch.empty(L, N, r, dtype=torch.bfloat16, device="cuda")
        ends = [torch.randn(2, r, K, generator=g).to(torch.bfloat16), torch.randn(2, N, r, generator=g).to(torch.bfloat16) / 8]
        for t, v in zip((a, b), ends):
            t[0], t[L - 1] = v[0].cuda(), v[1].cuda()
        x = torch.randn(M, K, generator=g).to(torch.bfloat16)
        ids = torch.where(torch.rand(M, generator=g) < 0.5, 0, L - 1).to(torch.int32)
        ids[0], ids[M - 1] = L - 1, 0
        out = _add(moe, a, b, None, x, ids, None, torch.float32)
        d, err = lora_delta(x, *ends, None, (ids > 0).to(torch.int32))
        check_rows(out, d, err, torch.float32)


def test_outputs_beyond_32_bits(moe):
    """Rows of out beyond 2^31 elements and 2^32 bytes, with and without the int8 projection."""
    g = torch.Generator().manual_seed(8)
    M, N, K, L, r = 14000, 157184, 16, 3, 8
    a, b, _ = _adapters(g, L, r, K, N, False)
    x, ids = torch.randn(M, K, generator=g).to(torch.bfloat16), torch.randint(-1, L, (M,), generator=g).to(torch.int32)
    lp, rows = moe.lora(a.cuda(), b.cuda()), [0, 1, 13660, 13663, M - 2, M - 1]
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = moe.lora_workspace(lp, M)
    moe.moe_lora_add(lp, x.cuda(), ids.cuda(), None, out, ws)
    d, err = lora_delta(x[rows], a, b, None, ids[rows])
    check_rows(out[rows], d, err, torch.bfloat16)
    q, w = (torch.randint(-127, 128, s, generator=g).to(torch.int8) for s in ((M, K), (N, K)))
    qs, wsc = torch.rand(M, generator=g) / 100, torch.rand(N, generator=g) / 100
    out.fill_(float("nan"))
    moe.moe_int8_linear_lora(q.cuda(), qs.cuda(), w.cuda(), wsc.cuda(), lp, x.cuda(), ids.cuda(), out, ws)
    base = (q[rows].double() @ w.double().T) * qs[rows].double()[:, None] * wsc.double()
    check_rows(out[rows], base + d, err + 2.0 ** -22 * base.abs(), torch.bfloat16)
