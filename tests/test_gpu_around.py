"""The operators around the expert layer together, as a decode step uses them:
norm -> routing by scores -> experts -> residual and norm -> int8 product; the
whole layer with routing by scores; captured into graphs, on other streams and
two at once.
"""
import numpy as np
import pytest
import torch

import oracle
from _around_gpu import Out, same_f32, up
from _around_ref import int8_product, int8_rows, rmsnorm, route
from _moe_helpers import DevWeights, dev, host, rel_l2
from mxfp4_weight_streaming_amd import synth

pytestmark = pytest.mark.gpu

BF, F32, I8, F8 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


@pytest.fixture(scope="module")
def ling():
    w = synth.expert_weights(1500, 2560, 768, 64)
    return w, DevWeights(w), synth.shared_expert(1501, 2560, 768)


def _router(moe, E, K):
    return moe.router(E, K, score="sigmoid", groups=8, group_topk=4, factor=2.5)


@pytest.mark.parametrize("M", [1, 2, 4, 8, 9, 17])
@pytest.mark.parametrize("shared", [False, True])
def test_scored_layer_is_its_parts(moe, ling, M, shared):
    """moe_decode_forward_scored gives the bits of the calls it stands for, and the oracle's layer."""
    w, dw, sh = ling
    H, I, E, K = 2560, 768, 64, 8
    shp, rp = moe.shape(H, I, E, K), _router(moe, E, K)
    rng = np.random.default_rng(1510 + M)
    x = synth.decode_tokens(1511 + M, w, M, K=K).x
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    dx, db = dev(x), up(bias)
    dsh = tuple(dev(t) for t in sh) if shared else None
    ws = moe.workspace(shp, M)
    out = Out((M, H), F32)
    moe.moe_decode_forward_scored(shp, rp, M, dx, dw.wr, db, dw.w13, dw.s13, dw.w2, dw.s2, out.t, ws, shared=dsh)
    logits, ids, tw = Out((M, E), F32), Out((M, K), torch.int32), Out((M, K), F32)
    q, s, parts = Out((M, H), torch.uint8), Out((M,), F32), Out((M, H), F32)
    moe.moe_router_logits(shp, M, dx, dw.wr, logits.t)
    moe.moe_route_scores(rp, logits.t, db, ids.t, tw.t)
    moe.moe_quant_act(shp, M, dx, q.t, s.t)
    moe.moe_experts_forward_shared(shp, M, q.t, s.t, ids.t, tw.t, dw.w13, dw.s13, dw.w2, dw.s2, dsh, parts.t, ws)
    torch.cuda.synchronize()
    assert same_f32(out.bits(), parts.bits())
    ri, rw = route(logits.bits(), bias, K, "sigmoid", 8, 4, 2, True, 2.5)
    assert np.array_equal(ids.bits(), ri)
    h = oracle.gate_up(q.bits(), s.bits(), ri, w.w13, w.s13, I)
    ref = oracle.down_combine(*oracle.requant(h), ri, rw, w.w2, w.s2, H)
    if shared:
        one = np.zeros((M, 1), np.int32)
        hs = oracle.gate_up(q.bits(), s.bits(), one, sh[0][None], sh[1][None], I)
        ref = ref + oracle.down_combine(*oracle.requant(hs), one, np.ones((M, 1)), sh[2][None], sh[3][None], H)
    assert rel_l2(out.bits(), ref) <= 1e-2


def test_scored_layer_on_the_one_kernel_path(moe, ling):
    w, dw, _ = ling
    H, I, E, K, M = 2560, 768, 64, 8, 3
    shp, rp = moe.shape(H, I, E, K), _router(moe, E, K)
    x = dev(synth.decode_tokens(1520, w, M, K=K).x)
    ws = moe.workspace(shp, 8)
    a, b = Out((M, H), F32), Out((M, H), F32)
    moe.moe_decode_forward_scored(shp, rp, M, x, dw.wr, None, dw.w13, dw.s13, dw.w2, dw.s2, a.t, ws)
    moe.moe_set_decode_path(moe.PATH_ONE_KERNEL)
    try:
        moe.moe_decode_forward_scored(shp, rp, M, x, dw.wr, None, dw.w13, dw.s13, dw.w2, dw.s2, b.t, ws)
    finally:
        moe.moe_set_decode_path(moe.PATH_THREE_KERNELS)
    torch.cuda.synchronize()
    assert moe.sync_errors(ws) == 0
    assert rel_l2(a.bits(), b.bits().astype(np.float64)) <= 1e-5


class Step:
    """One decode step's buffers: hidden comes from a norm, the layer's output goes through a norm into an int8 head."""

    def __init__(self, moe, dw, M, seed, V=1000):
        self.moe, self.dw, self.M = moe, dw, M
        rng = np.random.default_rng(seed)
        H, E, K = 2560, dw.E, 8
        self.np = dict(x=rng.standard_normal((M, H)).astype(np.float32),
                       res=synth.normal_bf16(rng, (M, H), 2.0),
                       w1=synth.bf16_from_f32((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)),
                       w2=synth.bf16_from_f32((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)),
                       bias=(0.1 * rng.standard_normal(E)).astype(np.float32),
                       head=synth.normal_bf16(rng, (V, H), 0.02))
        self.d = {k: up(v) for k, v in self.np.items()}
        self.shp, self.rp = moe.shape(H, 768, E, K), _router(moe, E, K)
        self.ws = moe.workspace(self.shp, max(M, 8))
        self.o = dict(r1=Out((M, H), BF), y1=Out((M, H), BF), q1=Out((M, H), F8), s1=Out((M,), F32),
                      lg=Out((M, E), F32), ids=Out((M, K), torch.int32), tw=Out((M, K), F32), out=Out((M, H), F32),
                      r2=Out((M, H), BF), q2=Out((M, H), I8), s2=Out((M,), F32), head_q=Out((V, H), I8),
                      head_s=Out((V,), F32), logits=Out((M, V), F32))
        moe.moe_int8_quantize(self.d["head"], self.o["head_q"].t, self.o["head_s"].t)

    def run(self, stream=None):
        moe, d, dw = self.moe, self.d, self.dw
        o = {k: v.t for k, v in self.o.items()}
        moe.moe_add_rmsnorm(d["x"], d["res"], d["w1"], 1e-6, o["r1"], y=o["y1"], q=o["q1"], scale=o["s1"], stream=stream)
        moe.moe_router_logits(self.shp, self.M, o["y1"], dw.wr, o["lg"], stream=stream)
        moe.moe_route_scores(self.rp, o["lg"], d["bias"], o["ids"], o["tw"], stream=stream)
        moe.moe_experts_forward(self.shp, self.M, o["q1"], o["s1"], o["ids"], o["tw"], dw.w13, dw.s13, dw.w2, dw.s2,
                                o["out"], self.ws, stream=stream)
        moe.moe_add_rmsnorm(o["out"], o["r1"], d["w2"], 1e-6, o["r2"], q=o["q2"], scale=o["s2"], stream=stream)
        moe.moe_int8_linear(o["q2"], o["s2"], o["head_q"], o["head_s"], o["logits"], stream=stream)

    def results(self):
        return {k: v.bits().copy() for k, v in self.o.items()}


@pytest.mark.parametrize("M", [1, 4, 12])
def test_a_step(moe, ling, M):
    """Each stage against its plain form on the bits the stage before it gave."""
    w, dw, _ = ling
    st = Step(moe, dw, M, 1530 + M)
    st.run()
    torch.cuda.synchronize()
    g, n = st.results(), st.np
    r1, y1, _ = rmsnorm(n["x"], n["res"], n["w1"], 1e-6, True)
    assert np.array_equal(g["r1"], r1) and np.array_equal(g["y1"], y1)
    q1, s1 = oracle.quant_act(y1)
    assert np.array_equal(g["q1"], q1) and same_f32(g["s1"], s1)
    ids, tw = route(g["lg"], n["bias"], 8, "sigmoid", 8, 4, 2, True, 2.5)
    assert np.array_equal(g["ids"], ids)
    h = oracle.gate_up(q1, s1, ids, w.w13, w.s13, 768)
    ref = oracle.down_combine(*oracle.requant(h), ids, tw, w.w2, w.s2, 2560)
    assert rel_l2(g["out"], ref) <= 1e-2
    r2, y2, _ = rmsnorm(g["out"], r1, n["w2"], 1e-6, True)
    q2, s2 = int8_rows(y2)
    assert np.array_equal(g["r2"], r2) and np.array_equal(g["q2"], q2) and same_f32(g["s2"], s2)
    hq, hs = int8_rows(n["head"])
    assert np.array_equal(g["head_q"], hq) and same_f32(g["head_s"], hs)
    assert same_f32(g["logits"], int8_product(q2, s2, hq, hs)[1])


@pytest.mark.parametrize("M", [1, 5, 40])
def test_graph_replays(moe, ling, M):
    """Two steps captured into two graphs, replayed with eager work between: every replay gives the eager bits."""
    _, dw, _ = ling
    steps = [Step(moe, dw, M, 1540 + M + k) for k in range(2)]
    for st in steps:
        st.run()
    torch.cuda.synchronize()
    ref = [st.results() for st in steps]
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
    for rep in range(3):
        for st in steps:
            for k in ("r1", "y1", "ids", "tw", "out", "logits"):
                st.o[k].t.view(torch.uint8).fill_(0xA5)
        for g in graphs if rep % 2 == 0 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for st, want in zip(steps, ref):
            got = st.results()
            for k in want:
                assert np.array_equal(got[k].view(np.uint8), want[k].view(np.uint8)), (rep, k)
        steps[rep % 2].run()                       # eager work on the same buffers between the replays
        _ = (a @ a).sum().item()


def test_two_streams_at_once(moe, ling):
    """Two steps on two streams without an order between them: the bits of each alone."""
    _, dw, _ = ling
    steps = [Step(moe, dw, m, 1550 + m) for m in (3, 40)]
    for st in steps:
        st.run()
    torch.cuda.synchronize()
    ref = [st.results() for st in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for st, s in zip(steps, streams):
            st.run(stream=s)
    torch.cuda.synchronize()
    for st, want in zip(steps, ref):
        got = st.results()
        for k in want:
            assert np.array_equal(got[k].view(np.uint8), want[k].view(np.uint8)), k
