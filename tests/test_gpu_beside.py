"""The log probabilities and the adapters as a decode step uses them: norm with
int8 codes -> int8 projection with adapters -> norm -> FP8 LM head -> its adapters
-> log probabilities of the drafted tokens; captured into graphs, on other
streams, two at once and with one workspace for everything.
"""
import numpy as np
import pytest
import torch

import oracle
from _around_gpu import Out, same_f32, up
from _around_ref import int8_product, int8_rows, rmsnorm
from _beside_ref import Logprobs, check_rows, lora_delta
from mxfp4_weight_streaming_amd import synth

pytestmark = pytest.mark.gpu

BF, F32, I8, F8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


class Step:
    """One step's buffers for M tokens of a few requests; one workspace serves every call of it in turn."""

    def __init__(self, moe, M, seed, H=512, V=3001, L=3, r=16, k=5):
        self.moe, self.M = moe, M
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.np = dict(x=rng.standard_normal((M, H)).astype(np.float32), res=synth.normal_bf16(rng, (M, H), 2.0),
                       w1=synth.bf16_from_f32((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)),
                       w2=synth.bf16_from_f32((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)),
                       proj=synth.normal_bf16(rng, (H, H), 0.05), head=synth.normal_bf16(rng, (V, H), 0.08))
        self.d = {n: up(v) for n, v in self.np.items()}
        self.ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
        self.tokens = torch.randint(0, V, (M,), generator=g).to(torch.int32)
        self.d["ids"], self.d["tokens"] = self.ids.cuda(), self.tokens.cuda()

        def adapters(N):
            a = (torch.randn(L, r, H, generator=g) / H ** 0.5).to(BF)
            b = (torch.randn(L, N, r, generator=g) / r ** 0.5).to(BF)
            return a, b, 0.5 + torch.rand(L, generator=g)

        self.proj_ad, self.head_ad = adapters(H), adapters(V)
        self.lp1, self.lp2 = (moe.lora(*(t.cuda() for t in ad)) for ad in (self.proj_ad, self.head_ad))
        self.ws = torch.empty(max(moe.lora_workspace(self.lp1, M).nbytes, moe.lora_workspace(self.lp2, M, product=False).nbytes,
                                  moe.logprobs_workspace(M, V, k).nbytes), dtype=torch.uint8, device="cuda")
        self.o = dict(r1=Out((M, H), BF), y1=Out((M, H), BF), q1=Out((M, H), I8), s1=Out((M,), F32), p=Out((M, H), BF),
                      r2=Out((M, H), BF), y2=Out((M, H), BF), head_logits=Out((M, V), F32), logits=Out((M, V), F32),
                      lp=Out((M,), F32), rank=Out((M,), torch.int32), ent=Out((M,), F32), top=Out((M, k), torch.int32),
                      toplp=Out((M, k), F32), pq=Out((H, H), I8), ps=Out((H,), F32), hq=Out((V, H), F8), hs=Out((V,), F32))
        moe.moe_int8_quantize(self.d["proj"], self.o["pq"].t, self.o["ps"].t)
        moe.moe_lm_head_quantize(self.d["head"], self.o["hq"].t, self.o["hs"].t)

    def run(self, stream=None):
        moe, d, ws = self.moe, self.d, self.ws
        o = {n: v.t for n, v in self.o.items()}
        moe.moe_add_rmsnorm(d["x"], d["res"], d["w1"], 1e-6, o["r1"], y=o["y1"], q=o["q1"], scale=o["s1"], stream=stream)
        moe.moe_int8_linear_lora(o["q1"], o["s1"], o["pq"], o["ps"], self.lp1, o["y1"], d["ids"], o["p"], ws, stream=stream)
        moe.moe_add_rmsnorm(o["p"], o["r1"], d["w2"], 1e-6, o["r2"], y=o["y2"], stream=stream)
        if self.M <= 8:
            moe.moe_lm_head_forward(o["y2"], o["hq"], o["hs"], o["head_logits"], stream=stream)
        else:
            moe.moe_lora_add(self.lp2, o["y2"], d["ids"], None, o["head_logits"], ws, stream=stream)
        moe.moe_lora_add(self.lp2, o["y2"], d["ids"], o["head_logits"], o["logits"], ws, stream=stream)
        moe.moe_token_logprobs(o["logits"], d["tokens"], o["lp"], o["rank"], o["ent"], o["top"], o["toplp"], ws, stream=stream)

    def results(self):
        return {n: v.bits().copy() for n, v in self.o.items()}


def _bf(bits):
    return torch.from_numpy(synth.bf16_to_f32(bits).astype(np.float32))


@pytest.mark.parametrize("M", [1, 4, 8, 20, 200, 600])
def test_a_step(moe, M):
    """Each stage against its plain form on the bits the stage before it gave."""
    st = Step(moe, M, 2000 + M)
    st.run()
    torch.cuda.synchronize()
    g, n = st.results(), st.np
    r1, y1, _ = rmsnorm(n["x"], n["res"], n["w1"], 1e-6, True)
    q1, s1 = int8_rows(y1)
    assert np.array_equal(g["r1"], r1) and np.array_equal(g["y1"], y1)
    assert np.array_equal(g["q1"], q1) and same_f32(g["s1"], s1)
    pq, ps = int8_rows(n["proj"])
    base = torch.from_numpy((q1.astype(np.float64) @ pq.astype(np.float64).T) * s1.astype(np.float64)[:, None] * ps.astype(np.float64))
    d, err = lora_delta(_bf(y1), *st.proj_ad, st.ids)
    check_rows(_bf(g["p"]), base + d, err + 2.0 ** -22 * base.abs(), BF)
    bare = (st.ids < 0).numpy()
    plain = synth.bf16_from_f32(int8_product(q1, s1, pq, ps)[1])
    assert np.array_equal(g["p"][bare], plain[bare])
    r2, y2, _ = rmsnorm(g["p"], r1, n["w2"], 1e-6, True)
    assert np.array_equal(g["r2"], r2) and np.array_equal(g["y2"], y2)
    d, err = lora_delta(_bf(y2), *st.head_ad, st.ids)
    if M <= 8:
        ref = oracle.lm_head_gemv(y2, g["hq"], g["hs"])
        assert np.max(np.abs(g["head_logits"] - ref)) <= 1e-4 * np.max(np.abs(ref))
    else:
        check_rows(g["head_logits"], d, err, F32)
    base = torch.from_numpy(g["head_logits"]).double()
    check_rows(g["logits"], base + d, err, F32)
    Logprobs(torch.from_numpy(g["logits"]), st.tokens, 5).check(g["lp"], g["rank"], g["ent"], g["top"], g["toplp"])


@pytest.mark.parametrize("M", [1, 4, 40, 600])
def test_graph_replays(moe, M):
    """Two steps captured into two graphs that share one workspace, replayed in turn with eager work between: every replay
    gives the eager bits."""
    steps = [Step(moe, M, 2100 + M + n) for n in range(2)]
    steps[1].ws = steps[0].ws
    ref = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        ref.append(st.results())
    graphs = []
    for st in steps:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            st.run()
        graphs.append(g)
    torch.cuda.synchronize()
    a = torch.randn(256, 256, device="cuda")
    for rep in range(4):
        for st in steps:
            for n in ("p", "head_logits", "logits", "lp", "rank", "ent", "top", "toplp"):
                st.o[n].t.view(torch.uint8).fill_(0xA5)
        steps[0].ws.fill_(0x5A + rep)
        for g in graphs if rep % 2 == 0 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for st, want in zip(steps, ref):
            got = st.results()
            for n in want:
                assert np.array_equal(got[n].view(np.uint8), want[n].view(np.uint8)), (rep, n)
        steps[rep % 2].run()                       # eager work on the same buffers between the replays
        _ = (a @ a).sum().item()


def test_two_streams_at_once(moe):
    """Two steps with a workspace each on two streams without an order between them: the bits of each alone."""
    steps = [Step(moe, m, 2200 + m) for m in (3, 70)]
    for st in steps:
        st.run()
    torch.cuda.synchronize()
    ref = [st.results() for st in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(8):
        for st, s in zip(steps, streams):
            st.run(stream=s)
    torch.cuda.synchronize()
    for st, want in zip(steps, ref):
        got = st.results()
        for n in want:
            assert np.array_equal(got[n].view(np.uint8), want[n].view(np.uint8)), n


@pytest.mark.parametrize("M", [3, 40, 600])
def test_int8_into_fp32_with_the_small_workspace(moe, M):
    """What the header says it needs is enough, and nothing behind it is written; the same bits as with a large one."""
    g = torch.Generator().manual_seed(M)
    L, r, K, N = 3, 40, 96, 300
    a, b = torch.randn(L, r, K, generator=g).to(BF).cuda(), torch.randn(L, N, r, generator=g).to(BF).cuda()
    lp = moe.lora(a, b)
    q, w = (torch.randint(-127, 128, s, generator=g).to(I8).cuda() for s in ((M, K), (N, K)))
    qs, ws = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    x, ids = torch.randn(M, K, generator=g).to(BF).cuda(), torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    small = moe.lora_workspace(lp, M, product=False)
    raw = torch.full((small.nbytes + 4096,), 0xC3, dtype=torch.uint8, device="cuda")
    outs = [Out((M, N), F32) for _ in range(2)]
    moe.moe_int8_linear_lora(q, qs, w, ws, lp, x, ids, outs[0].t, raw[:small.nbytes])
    moe.moe_int8_linear_lora(q, qs, w, ws, lp, x, ids, outs[1].t, moe.lora_workspace(lp, M))
    torch.cuda.synchronize()
    assert bool((raw[small.nbytes:] == 0xC3).all()) and same_f32(outs[0].bits(), outs[1].bits())
    d, err = lora_delta(x, a, b, None, ids)
    base = (q.cpu().double() @ w.cpu().double().T) * qs.cpu().double()[:, None] * ws.cpu().double()
    check_rows(outs[0].bits(), base + d, err + 2.0 ** -22 * base.abs(), F32)


def test_wide_rows_in_a_graph(moe):
    """Rows whose groups' maxima take more LDS than a kernel has by default, captured without an eager call before."""
    g = torch.Generator().manual_seed(11)
    M, V, k = 129, 270000, 2
    x, t = torch.randn(M, V, generator=g), torch.randint(0, V, (M,), generator=g).to(torch.int32)
    xd, td, o = x.cuda(), t.cuda(), [Out((M,), F32), Out((M,), torch.int32), Out((M,), F32), Out((M, k), torch.int32), Out((M, k), F32)]
    ws, graph = moe.logprobs_workspace(M, V, k), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        moe.moe_token_logprobs(xd, td, *(v.t for v in o), ws)
    ref = Logprobs(x, t, k)
    for _ in range(3):
        for v in o:
            v.t.view(torch.uint8).fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        ref.check(*(v.bits() for v in o))


def test_a_large_workspace_serves_fewer_tokens(moe):
    """A workspace for many tokens serves any smaller call; what a call does not use of it stays as it was."""
    V, k = 40000, 4
    ws = torch.full((moe.logprobs_workspace(128, V, k).nbytes,), 0xC3, dtype=torch.uint8, device="cuda")
    need = moe.logprobs_workspace(2, V, k).nbytes
    g = torch.Generator().manual_seed(5)
    x, t = torch.randn(2, V, generator=g), torch.randint(0, V, (2,), generator=g).to(torch.int32)
    o = [Out((2,), F32), Out((2,), torch.int32), Out((2,), F32), Out((2, k), torch.int32), Out((2, k), F32)]
    moe.moe_token_logprobs(x.cuda(), t.cuda(), *(v.t for v in o), ws)
    torch.cuda.synchronize()
    Logprobs(x, t, k).check(*(v.bits() for v in o))
    assert bool((ws[need:] == 0xC3).all())


def test_adapters_written_later_count(moe):
    """The description of adapters holds no values: weights swapped in place are used by the next call, a captured one too."""
    g = torch.Generator().manual_seed(6)
    L, r, K, N, M = 2, 8, 64, 96, 3
    mk = lambda: ((torch.randn(L, r, K, generator=g) / 8).to(BF), torch.randn(L, N, r, generator=g).to(BF), torch.rand(L, generator=g))  # noqa: E731
    first, second = mk(), mk()
    held = [t.cuda() for t in first]
    lp = moe.lora(*held)
    x, ids = torch.randn(M, K, generator=g).to(BF), torch.tensor([0, 1, 0], dtype=torch.int32)
    xd, idd, out, ws = x.cuda(), ids.cuda(), torch.empty(M, N, device="cuda"), moe.lora_workspace(lp, M)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_lora_add(lp, xd, idd, None, out, ws)
    for ad in (first, second, first):
        for t, v in zip(held, ad):
            t.copy_(v)
        for call in (lambda: moe.moe_lora_add(lp, xd, idd, None, out, ws), graph.replay):
            out.fill_(float("nan"))
            call()
            torch.cuda.synchronize()
            d, err = lora_delta(x, *ad, ids)
            check_rows(out, d, err, F32)


@pytest.mark.parametrize("M", [300, 513])
def test_int8_product_in_pieces(moe, M):
    """A product whose fp32 rows are kept in pieces (more rows than fit 256 MB, 256 at least) is the one of its rows alone."""
    N, K, L, r = 300000, 16, 2, 8
    g = torch.Generator().manual_seed(7)
    a, b = torch.randn(L, r, K, generator=g).to(BF).cuda(), (0.1 * torch.randn(L, N, r, generator=g)).to(BF).cuda()
    lp = moe.lora(a, b)
    q = torch.randint(-127, 128, (M, K), generator=g).to(I8).cuda()
    w = torch.randint(-127, 128, (N, K), generator=g).to(I8).cuda()
    qs, ws = torch.rand(M, generator=g).cuda() / 100, torch.rand(N, generator=g).cuda() / 100
    x, ids = torch.randn(M, K, generator=g).to(BF).cuda(), torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    out, part = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(40, N, dtype=BF, device="cuda")
    scratch = moe.lora_workspace(lp, M)
    assert scratch.nbytes < 320 << 20
    moe.moe_int8_linear_lora(q, qs, w, ws, lp, x, ids, out, scratch)
    for at in (0, 216, 240, M - 40):
        at = at // 8 * 8
        moe.moe_int8_linear_lora(q[at:at + 40], qs[at:at + 40], w, ws, lp, x[at:at + 40], ids[at:at + 40], part, scratch)
        # (the same sums in another order)
        ref, got = part.double(), out[at:at + 40].double()
        assert bool(((ref - got).abs() <= 2 * torch.finfo(BF).eps * ref.abs() + 1e-4).all())
