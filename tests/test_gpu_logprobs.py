"""moe_token_logprobs against sums in 64 bits: ids and ranks exactly, log
probabilities and entropies within the roundings of fp32 (tests/_beside_ref.py)."""
import numpy as np
import pytest
import torch

from _around_gpu import Out
from _beside_ref import Logprobs

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _logits(seed, M, V, dtype=torch.float32, pad=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(M, V + pad, generator=g)
    peak = torch.randint(V, (M, 1), generator=g)
    x.scatter_add_(1, peak, 30.0 * torch.rand(M, 1, generator=g))
    t = torch.where(torch.rand(M, generator=g) < 0.5, peak[:, 0], torch.randint(V, (M,), generator=g))
    return x.to(dtype)[:, :V], t.to(torch.int32)


def _run(moe, logits, tokens, k, stride_view=None):
    """The outputs on the GPU; logits may be a view of padded rows."""
    M, V = logits.shape
    outs = [Out((M,), torch.float32), Out((M,), torch.int32), Out((M,), torch.float32)]
    tops = [Out((M, k), torch.int32), Out((M, k), torch.float32)] if k else [None, None]
    ws = moe.logprobs_workspace(M, V, k)
    ws.fill_(0xFF)                                       # scratch: whatever stands in it
    moe.moe_token_logprobs(logits, tokens, *(o.t for o in outs), *(o and o.t for o in tops), ws)
    torch.cuda.synchronize()
    return [o and o.bits() for o in outs + tops]


def _check(moe, logits, tokens, k):
    dev = torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device="cuda")
    dev.copy_(logits)
    lp, rank, ent, ids, top = _run(moe, dev, tokens.cuda(), k)
    Logprobs(logits, tokens, max(k, 1)).check(lp, rank, ent, ids if k else None, top if k else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 31, 63, 64, 65, 255, 256, 257, 1000, 1023, 2049, 4097, 8191, 16385, 32771])
def test_vocabularies(moe, V, dtype):
    for M, k in ((1, 20), (3, 1), (17, 5), (5, 32), (2, 0)):
        print(f"V={V} M={M} k={k}", flush=True)
        _check(moe, *_logits(V * 7 + M + k, M, V, dtype), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,k", [(1, 157184, 20), (4, 157184, 1), (9, 157184, 32), (64, 40000, 5), (300, 5003, 3),
                                   (1025, 1000, 2), (2500, 130, 20), (1, 1000003, 7), (20, 262144, 0)])
def test_shapes(moe, M, V, k, dtype):
    print(f"M={M} V={V} k={k}", flush=True)
    _check(moe, *_logits(M + V + k, M, V, dtype), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,k", [(130, 262144, 32), (130, 300007, 2), (300, 30011, 9), (600, 20011, 4), (128, 16400, 3),
                                   (129, 16400, 3)])
def test_shapes_of_many_rows(moe, M, V, k, dtype):
    """Rows by 1,024, 512 and 256 threads, and on either side of where they are split."""
    print(f"M={M} V={V} k={k}", flush=True)
    _check(moe, *_logits(M + V + k, M, V, dtype), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,pad", [(1000, 1), (1000, 24), (1001, 2), (5003, 61), (40000, 7), (63, 1)])
def test_rows_apart(moe, V, pad, dtype):
    """Rows at any address; what lies between them is not read: it is NaN and +inf."""
    for M, k in ((1, 3), (6, 9), (70, 0)):
        x, t = _logits(V + pad + M, M, V, dtype, pad)
        full = torch.full((M, V + pad), INF, dtype=dtype)
        full[:, V::2] = float("nan")
        full[:, :V] = x
        _check(moe, full[:, :V], t, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9, 700, 5000, 40001, 157184])
def test_masks(moe, V, dtype):
    """Rows with most, all or all but a few logits masked, by -inf and by the type's lowest value; NaN counts as -inf."""
    g = torch.Generator().manual_seed(V)
    M = 12
    x, t = _logits(V, M, V, torch.float32)
    low = torch.finfo(dtype).min
    gone = torch.rand(M, V, generator=g) < 0.9
    x[0:4] = torch.where(gone[0:4], -INF, x[0:4])
    x[1] = torch.where(gone[1], low, x[1])
    x[2] = torch.where(torch.rand(V, generator=g) < 0.5, float("nan"), x[2])
    x[4] = -INF                                          # nothing left
    x[5] = low                                           # all alike, at the lowest value
    x[6] = float("nan")
    x[7] = -INF
    x[7, V // 2] = -4.0                                  # one left
    x[8] = -INF
    x[8, V - 1] = 3.0
    x[8, 0] = 3.0
    x[9] = low
    x[9, V // 3] = -INF
    x[10, 0] = low
    x = x.to(dtype)
    t[7] = V // 2
    t[9] = V // 3
    for k in (0, 1, 8, 32):
        _check(moe, x, t, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 300, 4100, 40001, 157184])
def test_ties_and_orders(moe, V, dtype):
    """Equal logits go to the lowest index, zeros of both signs alike; rows in rising and falling order, in steps and
    flat; a few values only."""
    g = torch.Generator().manual_seed(V + 1)
    ramp = torch.linspace(-8.0, 8.0, V)
    rows = [torch.zeros(V), torch.full((V,), 2.5), ramp, ramp.flip(0), torch.floor(ramp), -torch.floor(ramp).abs(),
            torch.randint(0, 3, (V,), generator=g).float(), torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0),
            (torch.arange(V) % 64).float(), (torch.arange(V) // 64 % 7).float(), -(torch.arange(V) % 1021).float(),
            torch.where(torch.arange(V) >= V - 2, 1.0, 0.0)]
    x = torch.stack(rows).to(dtype)
    t = torch.randint(0, V, (len(rows),), generator=g).to(torch.int32)
    t[0], t[1] = V - 1, 0
    for k in (1, 5, 32):
        _check(moe, x, t, k)


def test_infinities(moe):
    """+inf counts as the largest finite value, signalling NaNs as any NaN; distances beyond fp32's range."""
    big = torch.finfo(torch.float32).max
    V = 1000
    x = torch.randn(6, V, generator=torch.Generator().manual_seed(3))
    x[0, 17] = INF
    x[1, 17] = x[1, 400] = INF
    x[2, 5], x[2, 6] = INF, big
    x[3, 8], x[3, 9] = big, -big
    x[4, 10] = -big
    bits = x[5].view(torch.int32)
    bits[::3] = 0x7F800001                               # signalling NaN
    bits[1::9] = -0x7FFFFF                               # ... and a negative one
    t = torch.tensor([17, 400, 6, 9, 10, 2], dtype=torch.int32)
    for k in (1, 4):
        _check(moe, x, t, k)
    b = x[:4].to(torch.bfloat16)
    _check(moe, b, t[:4], 4)


def test_confident_rows(moe):
    """Log probabilities near 0 keep their digits: what stands beside the largest, down to 2^-100 of it."""
    V = 40000
    gap = torch.tensor([0.0, 1.0, 5.0, 12.0, 20.0, 30.0, 45.0, 60.0, 80.0])
    x = -gap[:, None] + 0.1 * torch.randn(len(gap), V, generator=torch.Generator().manual_seed(1))
    t = torch.arange(len(gap)) * 4321
    x[torch.arange(len(gap)), t] = 0.5
    _check(moe, x, t.to(torch.int32), 3)


@pytest.mark.parametrize("M,V", [(5, 300), (3, 157184), (40, 70)])
def test_tokens_outside(moe, M, V):
    """A token below 0 asks for nothing; one beyond the vocabulary has probability 0 and everything before it."""
    x, t = _logits(V, M, V)
    t[0], t[1], t[2] = -1, V, 2 ** 31 - 1
    if M > 3:
        t[3] = -2 ** 31
    _check(moe, x, t, 2)


def test_outputs_alone(moe):
    """Each output by itself is what it is beside the others."""
    for M, V, k in ((3, 157184, 6), (70, 1500, 6)):
        x, t = _logits(M, M, V)
        x, t = x.cuda(), t.cuda()
        lp, rank, ent, ids, top = _run(moe, x, t, k)
        ws = moe.logprobs_workspace(M, V, k)
        o = Out((M,), torch.float32)
        moe.moe_token_logprobs(x, t, logprob=o.t, ws=ws)
        assert np.array_equal(o.bits(), lp)
        o = Out((M,), torch.int32)
        moe.moe_token_logprobs(x, t, rank=o.t, ws=ws)
        assert np.array_equal(o.bits(), rank)
        o = Out((M,), torch.float32)
        moe.moe_token_logprobs(x, entropy=o.t, ws=ws)
        assert np.array_equal(o.bits(), ent)
        a, b = Out((M, k), torch.int32), Out((M, k), torch.float32)
        moe.moe_token_logprobs(x, topk_ids=a.t, topk_logprob=b.t, ws=ws)
        assert np.array_equal(a.bits(), ids) and np.array_equal(b.bits(), top)


def test_rows_do_not_depend_on_others(moe):
    """A row's ids and rank are the same in any batch (its sums may be split otherwise)."""
    V = 50001
    x, t = _logits(5, 600, V)
    x, t = x.cuda(), t.cuda()
    _, rank, _, ids, _ = _run(moe, x, t, 7)
    for at, n in ((0, 1), (3, 4), (100, 65), (590, 10)):
        _, r, _, i, _ = _run(moe, x[at:at + n].contiguous(), t[at:at + n].contiguous(), 7)
        assert np.array_equal(r, rank[at:at + n]) and np.array_equal(i, ids[at:at + n])


def test_offsets_beyond_32_bits(moe):
    """Rows that start beyond 2^31 elements and 2^32 bytes."""
    M, V, stride = 3, 50000, 1 << 30
    x, t = _logits(9, M, V, torch.bfloat16)
    store = torch.empty((M - 1) * stride + V, dtype=torch.bfloat16, device="cuda")
    rows = store.as_strided((M, V), (stride, 1))
    rows.copy_(x)
    lp, rank, ent, ids, top = _run(moe, rows, t.cuda(), 4)
    Logprobs(x, t, 4).check(lp, rank, ent, ids, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1024, 1025, 1100, 1500, 2047, 2048])
def test_rows_of_two_segments(moe, V, dtype):
    """Rows that a wave walks in two steps: sizes, distances, masks, ties."""
    test_vocabularies(moe, V, dtype)
    test_masks(moe, V, dtype)
    test_ties_and_orders(moe, V, dtype)
    test_rows_apart(moe, V, 3, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,pad", [(512, 2049, 0), (520, 3333, 5), (512, 4096, 0), (1024, 4097, 1), (1030, 6143, 2),
                                     (1024, 6144, 0)])
def test_many_rows_of_some_segments(moe, M, V, pad, dtype):
    """... and of up to six: many rows, plain ones beside flat, stepped, masked and empty ones."""
    print(f"M={M} V={V} pad={pad} {dtype}", flush=True)
    x, t = _logits(M + V, M, V, torch.float32)
    ramp = torch.linspace(-8.0, 8.0, V)
    odd = [torch.zeros(V), ramp, torch.floor(ramp), (torch.arange(V) % 64).float(), torch.full((V,), -INF), torch.full((V,), float("nan")),
           torch.where(torch.arange(V) == V - 1, 1.0, -INF), torch.where(torch.arange(V) >= V - 2, 1.0, 0.0),
           torch.where(torch.arange(V) % 3 == 0, float("nan"), -ramp), torch.full((V,), torch.finfo(dtype).min)]
    for i, row in enumerate(odd):
        for at in (i, M - 1 - i, M // 2 + i):
            x[at] = row
    full = torch.full((M, V + pad), INF, dtype=dtype)
    full[:, :V] = x.to(dtype)
    for k in (0, 3, 32):
        _check(moe, full[:, :V], t, k)
