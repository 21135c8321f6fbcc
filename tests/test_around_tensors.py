"""CPU-only checks of what the binding of the operators around the expert layer
refuses about tensors and streams, beyond tests/test_around_abi.py: said before
any device is asked for."""
from types import SimpleNamespace

import pytest
import torch

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
H, I, E, K, M = 256, 64, 16, 2, 3


@pytest.fixture
def moe(monkeypatch):
    """The binding, on a machine whose current device is 0; tensors on no GPU are on device -1."""
    from mxfp4_weight_streaming_amd import binding
    monkeypatch.setattr(binding, "_current", (lambda: 0, lambda d: 0))
    return binding


def test_router_logits_tensors(moe):
    good = dict(hidden=torch.zeros(M, H, dtype=BF), router_w=torch.zeros(E, H, dtype=BF), logits=torch.zeros(M, E))
    for bad in (dict(hidden=torch.zeros(M, H)), dict(hidden=torch.zeros(M - 1, H, dtype=BF)),
                dict(hidden=torch.zeros(H, M, dtype=BF).t()), dict(router_w=torch.zeros(E, H, dtype=torch.float16)),
                dict(router_w=torch.zeros(E, H - 32, dtype=BF)), dict(logits=torch.zeros(M, E, dtype=BF)),
                dict(logits=torch.zeros(M, E - 1)), dict(logits=torch.zeros(M, 2 * E)[:, ::2]),
                dict(logits=torch.zeros(M, E, device="meta"))):
        with pytest.raises(ValueError):
            moe.moe_router_logits(moe.shape(H, I, E, K), M, **{**good, **bad})


def _layer():
    return dict(hidden=torch.zeros(M, H, dtype=BF), router_w=torch.zeros(E, H, dtype=BF), bias=torch.zeros(E),
                w13=torch.zeros(E, 2 * I, H // 2, dtype=U8), w13_scale=torch.zeros(E, 2 * I, H // 32, dtype=U8),
                w2=torch.zeros(E, H, I // 2, dtype=U8), w2_scale=torch.zeros(E, H, I // 32, dtype=U8),
                out=torch.zeros(M, H), ws=torch.zeros(1 << 20, dtype=U8))


@pytest.mark.parametrize("name,bad", [
    ("bias", torch.zeros(E, dtype=torch.float64)), ("bias", torch.zeros(E, dtype=BF)), ("bias", torch.zeros(E - 1)),
    ("bias", torch.zeros(2 * E)[::2]),
    ("hidden", torch.zeros(M, H)), ("hidden", torch.zeros(M - 1, H, dtype=BF)),
    ("router_w", torch.zeros(E - 1, H, dtype=BF)), ("router_w", torch.zeros(H, E, dtype=BF).t()),
    ("w13", torch.zeros(E, I, H // 2, dtype=U8)), ("w13", torch.zeros(E, 2 * I, H // 2, dtype=torch.int16)),
    ("w13_scale", torch.zeros(E, 2 * I, H // 32)), ("w2", torch.zeros(E - 1, H, I // 2, dtype=U8)),
    ("w2_scale", torch.zeros(E, H // 2, I // 32, dtype=U8)),
    ("out", torch.zeros(M, H, dtype=BF)), ("out", torch.zeros(M, H - 1)), ("out", torch.zeros(H, M).t()),
    ("ws", torch.zeros(1 << 10, 2 << 10, dtype=U8)[:, ::2])])
def test_scored_layer_tensors(moe, name, bad):
    rp = moe.router(E, K, groups=4, group_topk=2)
    with pytest.raises(ValueError, match=name):
        moe.moe_decode_forward_scored(moe.shape(H, I, E, K), rp, M, **{**_layer(), name: bad})


@pytest.mark.parametrize("name", ["bias", "hidden", "router_w", "w13", "out", "ws"])
def test_scored_layer_tensor_on_no_device(moe, name):
    """A tensor without memory on the current device is refused, whichever it is."""
    bad = {name: _layer()[name].to("meta")}
    with pytest.raises(ValueError):
        moe.moe_decode_forward_scored(moe.shape(H, I, E, K), moe.router(E, K), M, **{**_layer(), **bad})


def test_scored_layer_shared_expert_tensors(moe):
    rp = moe.router(E, K, groups=4, group_topk=2)
    good = [torch.zeros(2 * I, H // 2, dtype=U8), torch.zeros(2 * I, H // 32, dtype=U8),
            torch.zeros(H, I // 2, dtype=U8), torch.zeros(H, I // 32, dtype=U8)]
    for shared in (good[:3], [good[0][:-1], *good[1:]], [*good[:3], good[3].float()],
                   [good[0], torch.zeros(2 * I, H // 16, dtype=U8)[:, ::2], *good[2:]]):
        with pytest.raises(ValueError):
            moe.moe_decode_forward_scored(moe.shape(H, I, E, K), rp, M, **_layer(), shared=shared)


def test_good_tensors_reach_the_device(moe):
    """What the documentation allows passes the tensors' checks: CPU tensors are refused for their device alone."""
    with pytest.raises(ValueError, match="current device"):
        moe.moe_decode_forward_scored(moe.shape(H, I, E, K), moe.router(E, K), M, **_layer())
    more = {**_layer(), "bias": None, "hidden": torch.zeros(M + 5, H, dtype=torch.int16), "out": torch.zeros(M + 5, H)}
    with pytest.raises(ValueError, match="current device"):
        moe.moe_decode_forward_scored(moe.shape(H, I, E, K), moe.router(E, K), M, **more)
    with pytest.raises(ValueError, match="current device"):
        moe.moe_router_logits(moe.shape(H, I, E, K), M, more["hidden"], more["router_w"], torch.zeros(M * E))


def test_route_scores_transposed_outputs(moe):
    """ids and weights come in rows of a token: tensors of as many elements with the tokens elsewhere are refused."""
    rp = moe.router(E, K)
    lg, ids, tw = torch.zeros(M, E), torch.empty(M, K, dtype=torch.int32), torch.empty(M, K)
    for bad in (dict(topk_ids=torch.empty(K, M, dtype=torch.int32)), dict(topk_w=torch.empty(K, M)),
                dict(topk_ids=torch.empty(1, M, K, dtype=torch.int32)), dict(topk_w=torch.empty(1, M * K)),
                dict(topk_ids=torch.tensor(0, dtype=torch.int32))):
        with pytest.raises(ValueError, match="topk_"):
            moe.moe_route_scores(rp, lg, None, **{**dict(topk_ids=ids, topk_w=tw), **bad})
    for good in (dict(), dict(topk_ids=ids.view(-1)), dict(topk_w=tw.view(M, 1, K)), dict(topk_w=tw.view(-1))):
        with pytest.raises(ValueError, match="current device"):
            moe.moe_route_scores(rp, lg, None, **{**dict(topk_ids=ids, topk_w=tw), **good})


def test_stream_of_another_device(moe, monkeypatch):
    """A stream of another device would run the kernel there, on this device's memory."""
    assert moe._stream_on(0, SimpleNamespace(device_index=0, cuda_stream=77)) == 77
    assert moe._stream_on(0, 78) == 78 and moe._stream_on(0, None) == 0
    with pytest.raises(ValueError, match="the stream on device 1"):
        moe._stream_on(0, SimpleNamespace(device_index=1, cuda_stream=77))
    # through a call: tensors on the (made up) current device, a stream of another
    monkeypatch.setattr(moe, "_current", (lambda: -1, lambda d: 0))
    with pytest.raises(ValueError, match="the stream on device 1"):
        moe.moe_route_scores(moe.router(E, K), torch.zeros(M, E), None, torch.empty(M, K, dtype=torch.int32),
                             torch.empty(M, K), stream=SimpleNamespace(device_index=1, cuda_stream=0))
