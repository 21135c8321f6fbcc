"""moe_token_logprobs on rows of every kind in every split of the work: masked by
-inf, by the type's lowest value and by others, flat, in steps, with equal
logits at their beginning and end, empty.  And what such rows cost."""
import numpy as np
import pytest
import torch

from _around_gpu import Out
from _beside_ref import Logprobs
from _beside_sizes import LOGPROB_ROWS, LOGPROB_SHORT_ROWS

pytestmark = pytest.mark.gpu

INF = float("inf")
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def kinds_of_rows(V, dtype, g):
    """Rows [n, V] of every kind, and a token of each."""
    at, ramp, low = torch.arange(V), torch.linspace(-8.0, 8.0, V), torch.finfo(dtype).min
    x = lambda: 3.0 * torch.randn(V, generator=g)  # noqa: E731
    few = lambda: torch.rand(V, generator=g) < 3.0 / V  # noqa: E731
    pick = lambda n: torch.randint(0, V, (n,), generator=g)  # noqa: E731
    rows = [x(), torch.where(torch.rand(V, generator=g) < 0.9, -INF, x()), torch.where(torch.rand(V, generator=g) < 0.9, low, x()),
            torch.where(few(), x(), low), torch.where(few(), x(), -1e9), torch.where(few(), x(), -INF),
            torch.where(torch.rand(V, generator=g) < 0.5, float("nan"), x()), torch.full((V,), -INF), torch.full((V,), float("nan")),
            torch.full((V,), low), torch.zeros(V), torch.where(at % 2 == 0, 0.0, -0.0), torch.where(at == V - 1, 3.0, -INF),
            ramp, ramp.flip(0), torch.floor(ramp), (at % 64).float(), (at // 64 % 7).float(), torch.randint(0, 3, (V,), generator=g).float(),
            torch.where(at >= V - 2, 1.0, 0.0), torch.where(at >= V - 700, 1.0, x() - 40.0), torch.full((V,), INF)]
    flat = torch.full((V,), -2.0)                        # fewer larger than any topk but 32, and the rest alike
    flat[pick(19)] = 1.0 + torch.arange(19.0) / 8
    rows.append(flat)
    for n in (22, 40):                                   # a few more left than 20 and 32, some of them in one lane's shares
        flat = torch.full((V,), torch.finfo(dtype).min)
        flat[pick(n)] = torch.randn(n, generator=g)
        rows.append(flat)
    # all logits of 24 threads' shares large (whatever the workgroup's size and type): more than are ranked at
    # once where a share is of two segments; the rest alike
    for threads, each in ((256, 4), (512, 4), (1024, 4), (256, 8), (512, 8), (1024, 8)):
        row, inside = torch.full((V,), -1.5), at % (16 * threads)
        row = torch.where((inside < 1024) & (inside // each % 64 < 24) & (at < 3 * 16 * threads), 1.0 + torch.rand(V, generator=g), row)
        rows.append(row)
    mixed = x()
    mixed[pick(3)], mixed[pick(3)], mixed[pick(40)] = INF, float("nan"), 30.0
    rows.append(mixed)
    t = torch.randint(0, V, (len(rows),), generator=g).to(torch.int32)
    t[3], t[9], t[10], t[20] = int(rows[3].argmax()), V - 1, V - 1, max(V - 350, 0)
    t[11] = -1
    return torch.stack(rows).to(dtype), t


def call(moe, x, t, k):
    M, V = x.shape
    outs = [Out((M,), torch.float32), Out((M,), torch.int32), Out((M,), torch.float32)]
    tops = [Out((M, k), torch.int32), Out((M, k), torch.float32)] if k else [None, None]
    ws = moe.logprobs_workspace(M, V, k)
    ws.fill_(0xFF)
    moe.moe_token_logprobs(x, t, *(o.t for o in outs), *(o and o.t for o in tops), ws)
    torch.cuda.synchronize()
    return [o and o.bits() for o in outs + tops]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V", LOGPROB_ROWS + LOGPROB_SHORT_ROWS)
def test_rows_of_every_kind(moe, M, V, dtype):
    """As many rows as the split of the work is for, of some 30 kinds in turn; equal rows give equal bits."""
    g = torch.Generator().manual_seed(M + V)
    rows, tokens = kinds_of_rows(V, dtype, g)
    n = len(rows)
    dev, dev_t = rows.cuda(), tokens.cuda()
    ref = Logprobs(rows, tokens, 32)
    for k in (0, 1, 20, 32):
        start = 0
        while start < n:                                 # (few rows: in several calls)
            which = (torch.arange(M) + start) % n
            print(f"M={M} V={V} k={k} {dtype} from {start}", flush=True)
            got = call(moe, dev[which.cuda()], dev_t[which.cuda()], k)
            first = {}
            for m, row in enumerate(which.tolist()):
                at = first.setdefault(row, m)
                for o in got:
                    assert o is None or at == m or np.array_equal(o[at].view(np.uint32), o[m].view(np.uint32)), (row, at, m)
            held = sorted(first)
            part = Logprobs.__new__(Logprobs)
            for name, v in vars(ref).items():
                setattr(part, name, v[held])
            lp, rank, ent, ids, top = (o if o is None else o[[first[r] for r in held]] for o in got)
            part.ids, part.top = part.ids[:, :k], part.top[:, :k]
            part.check(lp, rank, ent, ids, top)
            start += M


def _time(moe, x, k):
    M, V = x.shape
    t = torch.zeros(M, dtype=torch.int32, device="cuda")
    o = [torch.empty(M, device="cuda"), torch.empty(M, dtype=torch.int32, device="cuda"), torch.empty(M, device="cuda"),
         torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")]
    ws = moe.logprobs_workspace(M, V, k)
    run = lambda: moe.moe_token_logprobs(x, t, *o, ws)  # noqa: E731
    for _ in range(3):
        run()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            run()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


@pytest.mark.parametrize("M,V,k,dtype", [(1, 157184, 20, torch.float32), (64, 157184, 20, torch.float32), (64, 157184, 32, torch.bfloat16),
                                         (300, 32771, 32, torch.bfloat16), (600, 70001, 20, torch.float32), (16, 8192, 20, torch.float32)])
def test_a_finite_mask_costs_no_multiple(moe, M, V, k, dtype):
    """Rows whose excluded tokens hold a finite value, or that are flat, take a few times what those masked by -inf take at
    most, not topk times."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, V, generator=g, device="cuda")
    keep = torch.rand(M, V, generator=g, device="cuda") < 1e-4
    plain = _time(moe, torch.where(keep, x, -INF).to(dtype), k)
    for value in (torch.finfo(dtype).min, -1e9):
        masked = _time(moe, torch.where(keep, x, value).to(dtype), k)
        print(f"M={M} V={V} k={k} {dtype}: -inf {plain:.1f} us, {value} {masked:.1f} us", flush=True)
        assert masked < 5 * plain + 20
    flat = _time(moe, torch.zeros(M, V, dtype=dtype, device="cuda"), k)
    print(f"flat {flat:.1f} us", flush=True)
    assert flat < 5 * plain + 20


@pytest.mark.parametrize("M,V,dtype", [(1024, 6000, torch.float32), (512, 4096, torch.bfloat16), (1024, 2048, torch.float32)])
def test_a_finite_mask_of_short_rows_costs_no_multiple(moe, M, V, dtype):
    k = 32
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(M, V, generator=g, device="cuda")
    keep = torch.rand(M, V, generator=g, device="cuda") < 1e-3
    plain = _time(moe, torch.where(keep, x, -INF).to(dtype), k)
    for rows in (torch.where(keep, x, torch.finfo(dtype).min).to(dtype), torch.zeros(M, V, dtype=dtype, device="cuda")):
        masked = _time(moe, rows, k)
        print(f"M={M} V={V} {dtype}: -inf {plain:.1f} us, others {masked:.1f} us", flush=True)
        assert masked < 4 * plain
