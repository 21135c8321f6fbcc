"""CPU-only checks of the operators around the expert layer: every call refuses
what its documentation excludes, with the documented status, before anything
is enqueued, and the binding refuses tensors the calls cannot take."""
import ctypes

import pytest
import torch

A = 1 << 20          # an aligned address, never dereferenced: validation fails first
FAR = 1 << 40        # addresses that share no byte with A's buffers
FAR2 = 1 << 41
FAR3 = 1 << 42
FAR4 = 1 << 43


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _norm(moe, **k):
    v = dict(M=2, H=64, x=A, xt=1, res=FAR, rt=0, w=FAR2, wt=0, eps=1e-6, ro=FAR, y=FAR3, q=None, qt=0, s=None)
    v.update(k)
    return moe.raw().moe_add_rmsnorm(v["M"], v["H"], v["x"], v["xt"], v["res"], v["rt"], v["w"], v["wt"], v["eps"],
                                     v["ro"], v["y"], v["q"], v["qt"], v["s"], None)


@pytest.mark.parametrize("k,status", [
    (dict(M=0), -1), (dict(M=-1), -1), (dict(H=0), -1),
    (dict(H=32769), -2),
    (dict(x=None), -1), (dict(w=None), -1),
    (dict(xt=2), -1), (dict(rt=-1), -1), (dict(wt=5), -1),
    (dict(qt=3, q=FAR4, s=A), -1),
    (dict(qt=1), -1), (dict(q=FAR4), -1), (dict(s=FAR4), -1), (dict(qt=2, q=FAR4), -1), (dict(qt=2, s=FAR4), -1),
    (dict(ro=None, y=None), -1),
    (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(x=A + 4), -3), (dict(res=FAR + 8, ro=None), -3), (dict(w=FAR2 + 2), -3), (dict(y=FAR3 + 2), -3),
    (dict(ro=FAR4 + 4), -3), (dict(qt=1, q=FAR4 + 1, s=FAR4 + 4096), -3), (dict(qt=1, q=FAR4, s=FAR4 + 4097), -3),
    (dict(y=A), -1),                       # y over x
    (dict(y=A + 496), -1),                 # y over the end of x (2 * 64 * 4 bytes)
    (dict(y=FAR), -1),                     # y over residual_out
    (dict(ro=FAR + 16), -1),               # residual_out over residual, but not it
    (dict(ro=FAR2), -1),                   # residual_out over weight
    (dict(qt=1, q=FAR4, s=FAR4 + 16), -1),  # scale over q
])
def test_norm_refusals(moe, k, status):
    assert _norm(moe, **k) == status
    assert moe.moe_last_error() != ""


ROUTER = dict(num_experts=64, topk=8, score="sigmoid", groups=4, group_topk=2)


@pytest.mark.parametrize("change,status", [
    (dict(num_experts=0), -1), (dict(topk=0), -1), (dict(num_groups=0), -1), (dict(num_groups=5), -1),
    (dict(score=2), -1), (dict(score=-1), -1),
    (dict(group_topk=0), -1), (dict(group_topk=5), -1), (dict(group_score=0), -1), (dict(group_score=3), -1),
    (dict(num_groups=16, group_topk=1), -1),             # 8 of 4 experts
    (dict(num_experts=1024), -2), (dict(topk=9), -2), (dict(num_experts=512, num_groups=128, group_topk=8), -2),
    (dict(factor=float("inf")), -1), (dict(factor=float("nan")), -1),
])
def test_router_refusals(moe, change, status):
    rp = moe.router(**ROUTER)
    for k, v in change.items():
        setattr(rp, k, v)
    assert moe.raw().moe_route_scores(ctypes.byref(rp), 1, A, None, FAR, FAR2, None) == status
    shp = moe.shape(2560, 768, 64, 8)
    assert moe.raw().moe_decode_forward_scored(ctypes.byref(shp), ctypes.byref(rp), 1, A, A, None, A, A, A, A, None, A,
                                               A, 1 << 30, None) in (status, -1)


def test_route_scores_refusals(moe):
    L, rp = moe.raw(), moe.router(**ROUTER)
    r = ctypes.byref(rp)
    assert L.moe_route_scores(None, 1, A, None, FAR, FAR2, None) == -1
    assert L.moe_route_scores(r, 0, A, None, FAR, FAR2, None) == -1
    assert L.moe_route_scores(r, 1, None, None, FAR, FAR2, None) == -1
    assert L.moe_route_scores(r, 1, A, None, None, FAR2, None) == -1
    assert L.moe_route_scores(r, 1, A, None, FAR, None, None) == -1
    assert L.moe_route_scores(r, 1, A + 2, None, FAR, FAR2, None) == -3
    assert L.moe_route_scores(r, 1, A, A + 9, FAR, FAR2, None) == -3
    assert L.moe_route_scores(r, 1, A, None, FAR + 2, FAR2, None) == -3
    assert L.moe_route_scores(r, 1, A, None, FAR, FAR2 + 1, None) == -3
    assert L.moe_route_scores(r, 2, A, None, A + 508, FAR2, None) == -1     # ids over the end of the logits
    assert L.moe_route_scores(r, 2, A, None, FAR, FAR + 60, None) == -1     # weights over the end of the ids
    assert L.moe_route_scores(r, 2, A, FAR, FAR + 16, FAR2, None) == -1     # ids over the bias


def test_router_logits_and_scored_layer_refusals(moe):
    L = moe.raw()
    shp = moe.shape(2560, 768, 64, 8)
    s = ctypes.byref(shp)
    assert L.moe_router_logits(None, 1, A, FAR, FAR2, None) == -1
    assert L.moe_router_logits(s, 0, A, FAR, FAR2, None) == -1
    assert L.moe_router_logits(s, 2049, A, FAR, FAR2, None) == -2
    assert L.moe_router_logits(s, 1, None, FAR, FAR2, None) == -1
    assert L.moe_router_logits(s, 1, A, FAR + 2, FAR2, None) == -3
    assert L.moe_router_logits(s, 1, A, FAR, FAR2 + 4, None) == -3
    assert L.moe_router_logits(s, 1, A, FAR, A, None) == -1                 # logits over hidden
    need = moe.moe_workspace_bytes(shp, 4)
    rp = moe.router(**ROUTER)

    def call(M=4, rp=rp, hidden=A, bias=None, out=FAR, ws=FAR2, n=need):
        return L.moe_decode_forward_scored(s, ctypes.byref(rp), M, hidden, A, bias, A, A, A, A, None, out, ws, n, None)

    assert call(M=0) == -1
    assert call(hidden=None) == -1
    assert call(bias=A + 2) == -3
    assert call(out=None) == -1
    assert call(ws=None) == -4
    assert call(n=need - 1) == -4
    assert call(rp=moe.router(64, 4)) == -1                                  # another K than the shape's
    assert call(rp=moe.router(128, 8)) == -1                                 # another E


def test_int8_refusals(moe):
    L = moe.raw()
    assert L.moe_int8_quantize(None, 4, 64, FAR, FAR2, None) == -1
    assert L.moe_int8_quantize(A, 0, 64, FAR, FAR2, None) == -1
    assert L.moe_int8_quantize(A, 4, 0, FAR, FAR2, None) == -1
    assert L.moe_int8_quantize(A + 2, 4, 64, FAR, FAR2, None) == -3
    assert L.moe_int8_quantize(A, 4, 64, FAR + 1, FAR2, None) == -3
    assert L.moe_int8_quantize(A, 4, 64, FAR, FAR2 + 2, None) == -3
    assert L.moe_int8_quantize(A, 4, 64, A, FAR2, None) == -1                # codes over the input
    assert L.moe_int8_quantize(A, 4, 64, FAR, FAR + 252, None) == -1         # scales over the codes
    good = [A, FAR, FAR2, FAR3, 4, 64, 64, FAR4, 0, None]

    def call(at=None, v=None):
        args = list(good)
        if at is not None:
            args[at] = v
        return L.moe_int8_linear(*args)

    for at in (0, 1, 2, 3, 7):
        assert call(at, None) == -1
    for at in (4, 5, 6):
        assert call(at, 0) == -1
        assert call(at, -3) == -1
    assert call(6, 131072) == -2
    big = [1 << 44, FAR, 1 << 45, FAR2, 2 ** 31 - 1, 2 ** 31 - 1, 16, 1 << 50, 0, None]
    assert L.moe_int8_linear(*big) == -2                                     # beyond one launch's threads
    assert call(8, 2) == -1
    for at in (0, 2, 7):
        assert call(at, good[at] + 8) == -3
    for at in (1, 3):
        assert call(at, good[at] + 2) == -3
    assert call(7, A) == -1                                                  # out over a
    assert call(7, FAR2 + 4080) == -1                                        # out over the end of w


def test_binding_refuses_tensors(moe):
    """On CPU tensors: what is wrong with a tensor is said before any device is asked for."""
    x, w = torch.zeros(4, 64), torch.ones(64)
    out = torch.empty(4, 64)
    for bad in (dict(x=x.double()), dict(x=torch.zeros(64, 4).t()), dict(residual=torch.zeros(4, 63)),
                dict(residual=x.to(torch.bfloat16)), dict(weight=torch.ones(63)), dict(weight=w.half()),
                dict(residual_out=torch.empty(4, 128)[:, ::2]), dict(y=torch.empty(4, 64)),
                dict(q=torch.empty(4, 64, dtype=torch.float16)), dict(scale=torch.empty(3)),
                dict(scale=torch.empty(4, dtype=torch.float64))):
        k = dict(x=x, residual=x, weight=w, residual_out=out)
        k.update(bad)
        with pytest.raises(ValueError):
            moe.moe_add_rmsnorm(k.pop("x"), k.pop("residual"), k.pop("weight"), 1e-6, k.pop("residual_out"), **k)
    with pytest.raises(ValueError):
        moe.router(64, 8, score="tanh")
    rp = moe.router(**ROUTER)
    lg, ids, tw = torch.zeros(3, 64), torch.empty(3, 8, dtype=torch.int32), torch.empty(3, 8)
    for bad in (dict(logits=torch.zeros(3, 32)), dict(logits=lg.to(torch.bfloat16)), dict(bias=torch.zeros(63)),
                dict(topk_ids=ids.long()), dict(topk_ids=torch.empty(3, 7, dtype=torch.int32)),
                dict(topk_ids=torch.empty(3, 8)), dict(topk_w=torch.empty(3, 16)[:, ::2])):
        k = dict(logits=lg, bias=None, topk_ids=ids, topk_w=tw)
        k.update(bad)
        with pytest.raises(ValueError):
            moe.moe_route_scores(rp, **k)
    a, b = torch.zeros(3, 32, dtype=torch.int8), torch.zeros(5, 32, dtype=torch.int8)
    sa, sb, o = torch.ones(3), torch.ones(5), torch.empty(3, 5)
    for bad in (dict(a=a.float()), dict(a=a.to(torch.uint8)), dict(w=torch.zeros(5, 31, dtype=torch.int8)),
                dict(w=torch.zeros(32, 5, dtype=torch.int8).t()), dict(a_scale=torch.ones(4)),
                dict(w_scale=sb.double()), dict(out=torch.empty(5, 3)), dict(out=torch.empty(3, 5).half())):
        k = dict(a=a, a_scale=sa, w=b, w_scale=sb, out=o)
        k.update(bad)
        with pytest.raises(ValueError):
            moe.moe_int8_linear(**k)
    for q, s in ((torch.empty(3, 32), sa), (a, torch.ones(4))):
        with pytest.raises(ValueError):
            moe.moe_int8_quantize(torch.zeros(3, 32, dtype=torch.bfloat16), q, s)
