"""Tokens without an adapter: their rows are base's (or moe_int8_linear's) bit for bit, zeros' signs and NaNs' bits
included, whoever stands beside them."""
import numpy as np
import pytest
import torch

from _around_gpu import Out

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _bits(t):
    return t.cpu().contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


def _base(g, M, N, dtype):
    """Ordinary values among zeros of both signs, infinities, denormals and NaNs, quiet and signalling, of either sign."""
    y = torch.randn(M, N, generator=g).to(dtype)
    bits = y.view(torch.int32 if dtype == F32 else torch.int16)
    odd = [0x00000000, -0x80000000, 0x7F800000, -0x800000, 1, 0x7FC00000, -0x400000, 0x7F800001, 0x7F812345, -0x7EDCBB, 0x7FFFFFFF]
    if dtype == BF:
        odd = [0x0000, -0x8000, 0x7F80, -0x80, 1, 0x7FC0, -0x40, 0x7F81, 0x7FA3, -0x5D, 0x7FFF]
    which = torch.randint(0, 3 * len(odd), (M, N), generator=g)
    for i, v in enumerate(odd):
        bits[which == i] = v
    return y


def _bare(ids, L):
    return (ids < 0) | (ids >= L)


def _check(moe, M, L, r, K, N, dtype):
    print(f"M={M} L={L} r={r} K={K} N={N} {dtype}", flush=True)
    g = torch.Generator().manual_seed(M + r)
    a, b = torch.randn(L, r, K, generator=g).to(BF), torch.randn(L, N, r, generator=g).to(BF)
    lp = moe.lora(a.cuda(), b.cuda())
    x, y = torch.randn(M, K, generator=g).to(BF).cuda(), _base(g, M, N, dtype)
    for share in (0.5, 0.1, 0.0):                        # of tokens with an adapter; their neighbours in any order
        ids = torch.where(torch.rand(M, generator=g) < share, torch.randint(0, L, (M,), generator=g), -1).to(torch.int32)
        ids[torch.rand(M, generator=g) < 0.1] = L
        ids[0] = -1
        for in_place in (False, True):
            out = Out((M, N), dtype)
            src = y.cuda()
            if in_place:
                out.t.copy_(src)
                src = out.t
            moe.moe_lora_add(lp, x, ids.cuda(), src, out.t, moe.lora_workspace(lp, M))
            torch.cuda.synchronize()
            out.bits()
            bare = _bare(ids, L)
            assert torch.equal(_bits(out.t)[bare], _bits(y)[bare])
        out = Out((M, N), dtype)
        moe.moe_lora_add(lp, x, ids.cuda(), None, out.t, moe.lora_workspace(lp, M))
        torch.cuda.synchronize()
        assert bool((_bits(out.t)[bare] == 0).all())     # no base: zeros, +0


FEW = [(1, 2, 16, 64, 70), (5, 2, 8, 40, 33), (17, 3, 5, 72, 300), (40, 4, 64, 130, 65), (9, 3, 16, 9000, 130), (64, 3, 128, 96, 257),
       (3, 2, 12, 64, 9001)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,L,r,K,N", FEW)
def test_few_tokens(moe, M, L, r, K, N, dtype):
    _check(moe, M, L, r, K, N, dtype)


def _product(moe, M, L, r, K, N, dtype):
    print(f"M={M} L={L} r={r} K={K} N={N} {dtype}", flush=True)
    g = torch.Generator().manual_seed(M + r)
    a, b = torch.randn(L, r, K, generator=g).to(BF), torch.randn(L, N, r, generator=g).to(BF)
    lp = moe.lora(a.cuda(), b.cuda())
    x = torch.randn(M, K, generator=g).to(BF).cuda()
    q, w = (torch.randint(-127, 128, s, generator=g).to(torch.int8).cuda() for s in ((M, K), (N, K)))
    # scales of either sign, some so small that the product underflows to a zero of its sign, some infinite or NaN
    qs, ws = torch.randn(M, generator=g), torch.randn(N, generator=g)
    qs[::3] *= 1e-30
    ws[::2] *= 1e-25
    ws[1::7], ws[3::11] = torch.inf, torch.nan
    ids = torch.where(torch.rand(M, generator=g) < 0.4, torch.randint(0, L, (M,), generator=g), -1).to(torch.int32)
    ids[0] = -1
    dev = [q, qs.cuda(), w, ws.cuda()]
    out, plain = Out((M, N), dtype), Out((M, N), dtype)
    moe.moe_int8_linear_lora(*dev, lp, x, ids.cuda(), out.t, moe.lora_workspace(lp, M))
    moe.moe_int8_linear(*dev, plain.t)
    torch.cuda.synchronize()
    out.bits()
    bare = _bare(ids, L)
    want = _bits(plain.t)
    assert bool(((want & (0x7FFFFFFF if dtype == F32 else 0x7FFF)) == 0)[bare].any())      # (zeros, and negative ones)
    assert bool((want == (-0x80000000 if dtype == F32 else -0x8000))[bare].any())
    assert torch.equal(_bits(out.t)[bare], want[bare])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,L,r,K,N", FEW)
def test_few_tokens_with_the_product(moe, M, L, r, K, N, dtype):
    _product(moe, M, L, r, K, N, dtype)


# on the matrix cores: ranks of less than 8, of one, two and four steps, with and without slots
MANY = [(520, 3, 16, 64, 70), (520, 5, 3, 40, 33), (600, 20, 13, 72, 259), (300, 4, 64, 130, 65), (200, 3, 128, 96, 257), (2048, 40, 16, 64, 1030)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,L,r,K,N", MANY)
def test_many_tokens(moe, M, L, r, K, N, dtype):
    _check(moe, M, L, r, K, N, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,L,r,K,N", MANY)
def test_many_tokens_with_the_product(moe, M, L, r, K, N, dtype):
    _product(moe, M, L, r, K, N, dtype)
