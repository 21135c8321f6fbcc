"""The adapters' ways of splitting their work: on the matrix cores at every rank,
depth and number of channels that is read otherwise; u exactly; and what the
choice between one launch and two costs."""
import pytest
import torch

from _around_gpu import Out
from _beside_ref import check_rows, lora_delta
from _beside_sizes import LORA_CHANNELS, LORA_DEPTHS, LORA_LARGE, LORA_RANKS

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _ids(g, M, L):
    """Tokens in any order, requests one after another, and some without an adapter."""
    ids = torch.randint(-1, L, (M,), generator=g)
    half = M // 2
    ids[half:] = ids[half:half + (M - half + 10) // 11].repeat_interleave(11)[:M - half]
    ids[torch.rand(M, generator=g) < 0.05] = L
    return ids.to(torch.int32)


def _check(moe, M, r, K, N, dtype, base=True, scale=True, in_place=False, L=5):
    print(f"M={M} r={r} K={K} N={N} {dtype} base={base} scale={scale} in_place={in_place}", flush=True)
    g = torch.Generator().manual_seed(M + 7 * r + K + N)
    a, b = (torch.randn(L, r, K, generator=g) / K ** 0.5).to(BF), (torch.randn(L, N, r, generator=g) / r ** 0.5).to(BF)
    s = 0.5 + torch.rand(L, generator=g) if scale else None
    x, ids = torch.randn(M, K, generator=g).to(BF), _ids(g, M, L)
    y = torch.randn(M, N, generator=g).to(dtype) if base else None
    lp = moe.lora(a.cuda(), b.cuda(), None if s is None else s.cuda())
    ws = moe.lora_workspace(lp, M, product=False)
    ws.fill_(0xFF)
    out = Out((M, N), dtype)
    src = None if y is None else y.cuda()
    if in_place:
        out.t.copy_(src)
        src = out.t
    moe.moe_lora_add(lp, x.cuda(), ids.cuda(), src, out.t, ws)
    torch.cuda.synchronize()
    out.bits()
    d, err = lora_delta(x, a, b, s, ids)
    check_rows(out.t, d + (0 if y is None else y.double()), err, dtype)


@pytest.mark.parametrize("M,r,K,N", LORA_RANKS)
def test_ranks(moe, M, r, K, N):
    for dtype in (F32, BF):
        _check(moe, M, r, K, N, dtype)
        _check(moe, M, r, K, N, dtype, base=False)
        _check(moe, M, r, K, N, dtype, scale=False, in_place=True)


@pytest.mark.parametrize("M,r,K,N", LORA_DEPTHS)
def test_depths(moe, M, r, K, N):
    _check(moe, M, r, K, N, F32)


@pytest.mark.parametrize("M,r,K,N", LORA_CHANNELS)
def test_channels(moe, M, r, K, N):
    for dtype in (F32, BF):
        _check(moe, M, r, K, N, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,r,K,N", LORA_LARGE)
def test_many_tokens(moe, M, r, K, N, dtype):
    _check(moe, M, r, K, N, dtype)
    _check(moe, M, r, K, N, dtype, L=300)


@pytest.mark.parametrize("M,r,K,N", LORA_RANKS[::2] + LORA_DEPTHS[::3] + LORA_CHANNELS[::4] + LORA_LARGE)
def test_with_the_int8_product(moe, M, r, K, N):
    L = 5
    g = torch.Generator().manual_seed(M + r + K + N)
    a, b = (torch.randn(L, r, K, generator=g) / K ** 0.5).to(BF), (torch.randn(L, N, r, generator=g) / r ** 0.5).to(BF)
    s, x, ids = 0.5 + torch.rand(L, generator=g), torch.randn(M, K, generator=g).to(BF), _ids(g, M, L)
    q, w = (torch.randint(-127, 128, n, generator=g).to(torch.int8) for n in ((M, K), (N, K)))
    qs, ws = (0.01 + torch.rand(M, generator=g)) / K ** 0.5 / 50, (0.01 + torch.rand(N, generator=g)) / 50
    lp = moe.lora(a.cuda(), b.cuda(), s.cuda())
    base = (q.double() @ w.double().t()) * qs.double()[:, None] * ws.double()
    d, err = lora_delta(x, a, b, s, ids)
    for dtype in (F32, BF):
        print(f"M={M} r={r} K={K} N={N} {dtype}", flush=True)
        out, scratch = Out((M, N), dtype), moe.lora_workspace(lp, M)
        scratch.fill_(0xFF)
        moe.moe_int8_linear_lora(q.cuda(), qs.cuda(), w.cuda(), ws.cuda(), lp, x.cuda(), ids.cuda(), out.t, scratch)
        torch.cuda.synchronize()
        out.bits()
        # (the product's own two roundings, of its value and not of the sum's)
        check_rows(out.t, base + d, err + 2.0 ** -22 * base.abs(), dtype)


def _three_parts(v):
    """fp32 values as three bf16 numbers that add up to them, each the 8 leading bits of what is left."""
    parts = []
    for _ in range(3):
        parts.append((v.view(torch.int32) & -65536).view(F32))
        v = v - parts[-1]
    assert bool((v == 0).all())
    return parts


@pytest.mark.parametrize("M", [1, 9, 40, 140, 270, 530])
@pytest.mark.parametrize("r", [5, 8, 13, 16, 24, 29, 32, 40, 61, 64, 90, 96, 127, 128])
def test_u_is_not_rounded(moe, M, r):
    """x has the three parts of a value of 24 bits, A their sum times a power of two, and a channel of B one rank times a
    power of two: every sum is exact in any order, so the output has all 24 bits of u, or an error is in sight.  (Without
    u's last 8 bits nearly every value would differ.)"""
    g = torch.Generator().manual_seed(M + r)
    L, K, N = 3, 200, 3 * r + 1
    pick = lambda n, *s: torch.randint(0, n, s, generator=g)  # noqa: E731
    power = lambda *s: torch.ldexp(1.0 - 2.0 * pick(2, *s), pick(9, *s) - 4)  # noqa: E731
    v = torch.randn(M, generator=g)
    h, m, l = _three_parts(v)
    assert float((l != 0).float().mean()) > 0.9 or M < 40
    ids = pick(L, M)
    a, b, x = torch.zeros(L, r, K), torch.zeros(L, N, r), torch.randn(M, K, generator=g)
    ups = power(L, r)
    for i in range(L):
        at = torch.randperm(K, generator=g)[:3]
        a[i][:, at] = ups[i][:, None].expand(r, 3)
        rows = ids == i
        for p, part in zip(at.tolist(), (h, m, l)):
            x[rows, p] = part[rows]
    rank = torch.arange(N) % r
    downs = power(L, N)
    b[:, torch.arange(N), rank] = downs
    scale = torch.tensor([1.0, 0.5, -4.0])
    want = v[:, None] * scale[ids][:, None] * ups[ids][:, rank] * downs[ids]      # (only powers of two: exact)
    lp = moe.lora(a.to(BF).cuda(), b.to(BF).cuda(), scale.cuda())
    assert torch.equal(a.to(BF).float(), a) and torch.equal(b.to(BF).float(), b)
    xb, idd, ws = x.to(BF).cuda(), ids.to(torch.int32).cuda(), moe.lora_workspace(lp, M)
    out = Out((M, N), F32)
    moe.moe_lora_add(lp, xb, idd, None, out.t, ws)
    torch.cuda.synchronize()
    out.bits()
    assert torch.equal(out.t.cpu(), want)
    zero = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
    w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    out = Out((M, N), F32)
    moe.moe_int8_linear_lora(*zero, *w, lp, xb, idd, out.t, ws)
    torch.cuda.synchronize()
    assert torch.equal(out.t.cpu(), want)


@pytest.mark.parametrize("r", [3, 13, 16, 40, 128])
@pytest.mark.parametrize("M", [12, 60, 200, 600, 1100])
def test_a_row_does_not_depend_on_its_place(moe, M, r):
    """Tokens that occur several times among others give the same bits everywhere."""
    g = torch.Generator().manual_seed(M + r)
    L, K, N = 4, 300, 131
    lp = moe.lora(torch.randn(L, r, K, generator=g).to(BF).cuda(), torch.randn(L, N, r, generator=g).to(BF).cuda(),
                  torch.rand(L, generator=g).cuda())
    x, ids, y = torch.randn(M, K, generator=g).to(BF), _ids(g, M, L), torch.randn(M, N, generator=g)
    q = torch.randint(-127, 128, (M, K), generator=g).to(torch.int8)
    qs, w, ws = torch.rand(M, generator=g), torch.randint(-127, 128, (N, K), generator=g).to(torch.int8), torch.rand(N, generator=g)
    source = torch.where(torch.rand(M, generator=g) < 0.5, torch.randint(0, 5, (M,), generator=g), torch.arange(M))
    source[:5] = torch.arange(5)                         # (those that are repeated are themselves)
    x, ids, y, q, qs = (t[source].cuda() for t in (x, ids, y, q, qs))
    scratch = moe.lora_workspace(lp, M)
    for dtype in (F32, BF):
        out = torch.empty(M, N, dtype=dtype, device="cuda")
        moe.moe_lora_add(lp, x, ids, y.to(dtype), out, scratch)
        assert torch.equal(out, out[source.cuda()])
        moe.moe_int8_linear_lora(q, qs, w.cuda(), ws.cuda(), lp, x, ids, out, scratch)
        assert torch.equal(out, out[source.cuda()])


def test_a_row_does_not_depend_on_its_piece(moe):
    """Rows of the int8 product that are taken some at a time: the last, fewer ones as the others."""
    g = torch.Generator().manual_seed(9)
    M, N, K, L, r = 520, 300000, 24, 3, 8                # 256, 256 and 8 rows
    lp = moe.lora(torch.randn(L, r, K, generator=g).to(BF).cuda(), torch.randn(L, N, r, generator=g).to(BF).cuda())
    q, w = (torch.randint(-127, 128, s, generator=g).to(torch.int8).cuda() for s in ((M, K), (N, K)))
    qs, ws = torch.rand(M, generator=g).cuda() / 1000, torch.rand(N, generator=g).cuda() / 1000
    x, ids = torch.randn(M, K, generator=g).to(BF).cuda(), torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    for t in (q, qs, x, ids):
        t[512:] = t[:8]
    out = torch.empty(M, N, dtype=BF, device="cuda")
    moe.moe_int8_linear_lora(q, qs, w, ws, lp, x, ids, out, moe.lora_workspace(lp, M))
    assert torch.equal(out[512:], out[:8])


def _time(moe, M, r, K, N):
    """Microseconds of a call in a graph, an adapter a token."""
    g = torch.Generator(device="cuda").manual_seed(M)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    lp = moe.lora(draw(M, r, K), draw(M, N, r))
    x, y, ids = draw(M, K), draw(M, N), torch.arange(M, dtype=torch.int32, device="cuda")
    out, ws = torch.empty(M, N, dtype=BF, device="cuda"), moe.lora_workspace(lp, M)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(40):
            moe.moe_lora_add(lp, x, ids, y, out, ws)
    best = float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 25)
    return best


@pytest.mark.parametrize("K,M", [(8192, 24), (2560, 48)])
def test_a_few_tokens_more_cost_little(moe, K, M):
    """No step in time from a number of tokens that the XCDs share evenly to one that they do not."""
    even, odd = _time(moe, M, 16, K, 2560), _time(moe, M + 1 if K > 2560 else M + 3, 16, K, 2560)
    print(f"K={K}: {M} tokens {even:.2f} us, the odd number {odd:.2f} us", flush=True)
    assert odd < 1.3 * even
