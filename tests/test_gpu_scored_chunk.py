"""moe_decode_forward_scored on chunks of tokens: the bits of the calls it
stands for, whose stages tests/test_gpu_chunk.py and
tests/test_gpu_route_scores.py hold to their references; and in a graph."""
import numpy as np
import pytest
import torch

from _around_gpu import Out, same_f32, up
from _moe_helpers import DevWeights, dev
from mxfp4_weight_streaming_amd import synth

pytestmark = pytest.mark.gpu

F32 = torch.float32
H, I, E, K = 2560, 768, 64, 8


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


@pytest.fixture(scope="module")
def ling():
    w = synth.expert_weights(1600, H, I, E)
    return DevWeights(w), tuple(dev(t) for t in synth.shared_expert(1601, H, I))


def _inputs(M):
    rng = np.random.default_rng(1610 + M)
    return dev(synth.normal_bf16(rng, (M, H), 1.0)), up((0.1 * rng.standard_normal(E)).astype(np.float32))


def _parts(moe, shp, rp, M, x, bias, dw, shared, ws):
    logits, ids, tw = Out((M, E), F32), Out((M, K), torch.int32), Out((M, K), F32)
    q, s, out = Out((M, H), torch.uint8), Out((M,), F32), Out((M, H), F32)
    moe.moe_router_logits(shp, M, x, dw.wr, logits.t)
    moe.moe_route_scores(rp, logits.t, bias, ids.t, tw.t)
    moe.moe_quant_act(shp, M, x, q.t, s.t)
    moe.moe_experts_forward_shared(shp, M, q.t, s.t, ids.t, tw.t, dw.w13, dw.s13, dw.w2, dw.s2, shared, out.t, ws)
    torch.cuda.synchronize()
    return out.bits().copy()


@pytest.mark.parametrize("M", [33, 512, 1001, 2048])
@pytest.mark.parametrize("with_shared", [False, True])
def test_chunk_is_its_parts(moe, ling, M, with_shared):
    dw, sh = ling
    shared = sh if with_shared else None
    shp, rp = moe.shape(H, I, E, K), moe.router(E, K, score="sigmoid", groups=8, group_topk=4, factor=2.5)
    x, bias = _inputs(M)
    ws = moe.workspace(shp, M)
    want = _parts(moe, shp, rp, M, x, bias, dw, shared, ws)
    assert np.isfinite(want).all() and want.any(1).all()
    out = Out((M, H), F32)
    args = (shp, rp, M, x, dw.wr, bias, dw.w13, dw.s13, dw.w2, dw.s2, out.t, ws)
    moe.moe_decode_forward_scored(*args, shared=shared)
    torch.cuda.synchronize()
    assert same_f32(out.bits(), want)
    # captured and replayed, with other work of the program on the workspace between
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        moe.moe_decode_forward_scored(*args, shared=shared)
    for _ in range(3):
        out.t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same_f32(out.bits(), want)
        assert same_f32(_parts(moe, shp, rp, M, x, bias, dw, shared, ws), want)
