"""CPU-only checks of the log probabilities and the adapters: every call
refuses what its documentation excludes, with the documented status, before
anything is enqueued, and the binding refuses tensors the calls cannot take."""
import ctypes

import pytest
import torch

A = 1 << 20          # aligned addresses, never dereferenced: validation fails first
B, C, D, E, F, G, H, I = (1 << n for n in range(40, 48))


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _logprobs(moe, **k):
    v = dict(M=2, V=64, logits=A, type=1, stride=64, tokens=B, logprob=C, rank=D, entropy=E, topk=4, ids=F, top=G, ws=H,
             n=1 << 30)
    v.update(k)
    return moe.raw().moe_token_logprobs(v["M"], v["V"], v["logits"], v["type"], v["stride"], v["tokens"], v["logprob"],
                                        v["rank"], v["entropy"], v["topk"], v["ids"], v["top"], v["ws"], v["n"], None)


@pytest.mark.parametrize("k,status", [
    (dict(M=0), -1), (dict(M=-1), -1), (dict(V=0), -1), (dict(V=-5), -1), (dict(logits=None), -1),
    (dict(type=2), -1), (dict(type=-1), -1), (dict(stride=63), -1), (dict(stride=-64), -1), (dict(stride=(1 << 30) + 1), -1),
    (dict(tokens=None), -1), (dict(logprob=None, rank=None), -1),
    (dict(topk=-1), -1), (dict(topk=0), -1), (dict(topk=0, ids=None), -1), (dict(ids=None), -1), (dict(top=None), -1),
    (dict(topk=0, ids=None, top=None, tokens=None, logprob=None, rank=None, entropy=None), -1),
    (dict(topk=33), -2),
    (dict(logits=A + 2), -3), (dict(logits=A + 1, type=0), -3), (dict(tokens=B + 2), -3), (dict(logprob=C + 1), -3), (dict(rank=D + 2), -3),
    (dict(entropy=E + 3), -3), (dict(ids=F + 2), -3), (dict(top=G + 1), -3),
    (dict(logprob=A), -1), (dict(logprob=A + 508), -1),  # over the logits, over their end (2 * 64 * 4 bytes)
    (dict(rank=B + 4), -1),                              # over the tokens
    (dict(entropy=C + 4), -1), (dict(ids=D), -1), (dict(top=F + 28), -1),
    (dict(stride=1000, entropy=A + 4000 + 252), -1),     # over the end of rows that stand apart
    (dict(V=1 << 20, stride=1 << 20, M=1, ws=None), -4), (dict(V=1 << 20, stride=1 << 20, M=1, ws=H + 16), -4),
    (dict(V=1 << 20, stride=1 << 20, M=1, n=8), -4), (dict(V=1 << 20, stride=1 << 20, M=1, ws=F), -1),
])
def test_logprobs_refusals(moe, k, status):
    if ("ws" in k or "n" in k) and moe.raw().moe_token_logprobs_workspace_bytes(1, 1 << 20, 4) == 0:
        pytest.skip("these sizes take no workspace")
    assert _logprobs(moe, **k) == status
    assert moe.moe_last_error() != ""


def test_workspace_sizes(moe):
    n = moe.raw().moe_token_logprobs_workspace_bytes
    assert n(0, 10, 1) == n(1, 0, 1) == n(1, 10, -1) == n(1, 10, 33) == 0
    for V in (1, 1000, 157184, 1 << 22):
        for k in (0, 1, 32):
            sizes = [n(M, V, k) for M in (1, 2, 3, 8, 64, 255, 256, 257, 1000, 5000)]
            assert sizes == sorted(sizes)                # what serves many rows serves fewer
    lora = moe.MoeLora(4, 16, 64, 96, A, B, None)
    n = moe.raw().moe_lora_workspace_bytes
    assert n(None, 4) == n(ctypes.byref(lora), 0) == 0
    sizes = [n(ctypes.byref(lora), M) for M in (1, 2, 7, 64, 1000, 5000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("M,r", [(1, 1), (2, 16), (3, 33), (64, 128), (1000, 40)])
def test_adding_adapters_needs_their_u_alone(moe, M, r):
    lp = moe.MoeLora(4, r, 64, 96, A, B, None)
    need = M * ((r + 31) // 32 * 32) * 4
    need = (need + 255) // 256 * 256
    assert need < moe.raw().moe_lora_workspace_bytes(ctypes.byref(lp), M)
    # (one byte less is refused; as much is enough, so that the overlap of the workspace's first byte is what is)
    call = lambda ws, n: moe.raw().moe_lora_add(ctypes.byref(lp), M, D, E, None, G, 0, ws, n, None)  # noqa: E731
    assert call(H, need - 1) == -4 and "workspace" in moe.moe_last_error()
    assert call(D, need) == -1 and "overlap" in moe.moe_last_error()
    # the int8 projection into fp32 as well; into bf16 it keeps its product in the workspace, too
    call = lambda ws, n, kind: moe.raw().moe_int8_linear_lora(  # noqa: E731
        D, E, F, G, ctypes.byref(lp), M, H, I, 1 << 48, kind, ws, n, None)
    assert call(1 << 49, need - 1, 1) == -4 and call(1 << 48, need, 1) == -1 and call(1 << 49, need, 0) == -4


LORA = dict(L=4, r=16, K=64, N=96, a=A, b=B, s=C)


def _lora(moe, **k):
    v = {**LORA, **k}
    return moe.MoeLora(v["L"], v["r"], v["K"], v["N"], v["a"], v["b"], v["s"])


BAD_LORA = [(dict(L=0), -1), (dict(r=0), -1), (dict(K=0), -1), (dict(N=0), -1), (dict(L=-1), -1), (dict(a=None), -1),
            (dict(b=None), -1), (dict(r=129), -2), (dict(L=65536), -2), (dict(K=(1 << 24) + 1), -2), (dict(a=A + 2), -3), (dict(b=B + 8), -3),
            (dict(s=C + 2), -3)]


@pytest.mark.parametrize("k,status", BAD_LORA)
def test_adapter_refusals(moe, k, status):
    lp = _lora(moe, **k)
    L = moe.raw()
    assert L.moe_lora_workspace_bytes(ctypes.byref(lp), 4) == 0
    assert L.moe_lora_add(ctypes.byref(lp), 2, D, E, F, G, 0, H, 1 << 30, None) == status
    assert L.moe_int8_linear_lora(D, E, F, G, ctypes.byref(lp), 2, H, I, 1 << 48, 0, 1 << 49, 1 << 30, None) == status


@pytest.mark.parametrize("k,status", [
    (dict(M=0), -1), (dict(M=-2), -1), (dict(x=None), -1), (dict(ids=None), -1), (dict(out=None), -1),
    (dict(type=2), -1), (dict(x=D + 2), -3), (dict(ids=E + 1), -3), (dict(base=F + 8), -3), (dict(out=G + 4), -3),
    (dict(ws=None), -4), (dict(ws=H + 128), -4), (dict(n=16), -4),
    (dict(out=D), -1), (dict(out=E), -1), (dict(out=A), -1), (dict(out=B), -1), (dict(out=C), -1),
    (dict(out=F + 16), -1),                              # over a part of base
    (dict(out=A + 4 * 16 * 64 * 2 - 16), -1),            # over the end of the adapters
    (dict(ws=D), -1), (dict(ws=F), -1), (dict(ws=F, out=F), -1), (dict(ws=G), -1), (dict(ws=A), -1),
])
def test_lora_add_refusals(moe, k, status):
    v = dict(M=2, x=D, ids=E, base=F, out=G, type=0, ws=H, n=1 << 20)
    v.update(k)
    lp = _lora(moe)
    assert moe.raw().moe_lora_add(ctypes.byref(lp), v["M"], v["x"], v["ids"], v["base"], v["out"], v["type"], v["ws"], v["n"],
                                  None) == status
    assert moe.moe_last_error() != ""
    assert moe.raw().moe_lora_add(None, 2, D, E, F, G, 0, H, 1 << 20, None) == -1


def test_int8_linear_lora_refusals(moe):
    L, lp = moe.raw(), _lora(moe)
    good = [D, E, F, G, ctypes.byref(lp), 2, H, I, 1 << 48, 0, 1 << 49, 1 << 20, None]

    def call(at, v):
        args = list(good)
        args[at] = v
        return L.moe_int8_linear_lora(*args)

    for at in (0, 1, 2, 3, 4, 6, 7, 8):
        assert call(at, None) == -1
    assert call(5, 0) == call(5, -1) == call(9, 2) == -1
    for at in (0, 2, 6, 8):
        assert call(at, good[at] + 8) == -3
    for at in (1, 3, 7):
        assert call(at, good[at] + 2) == -3
    assert call(10, None) == call(10, good[10] + 64) == call(11, 8) == -4
    for v in (A, B, C, D, E, F, G, H, I):
        assert call(8, v) == -1                          # out over an input
        assert call(10, v) == -1                         # the workspace over one
    assert call(10, good[8]) == -1
    deep = _lora(moe, K=131072)
    assert call(4, ctypes.byref(deep)) == -2
    wide = _lora(moe, N=2 ** 31 - 1)
    args = list(good)
    args[4], args[5], args[8], args[10], args[11] = ctypes.byref(wide), 2 ** 31 - 1, 1 << 52, 1 << 62, 1 << 61
    assert L.moe_int8_linear_lora(*args) in (-1, -2)     # beyond one launch's threads


def test_binding_refuses_tensors(moe):
    """On CPU tensors: what is wrong with a tensor is said before any device is asked for."""
    M, V, k = 3, 50, 4
    i32 = torch.int32
    good = dict(logits=torch.zeros(M, V), tokens=torch.zeros(M, dtype=i32), logprob=torch.empty(M), rank=torch.empty(M, dtype=i32),
                entropy=torch.empty(M), topk_ids=torch.empty(M, k, dtype=i32), topk_logprob=torch.empty(M, k))
    for bad in (dict(logits=torch.zeros(V, M).t()), dict(logits=torch.zeros(M, 2 * V)[:, ::2]),
                dict(logits=torch.zeros(M, V).double()), dict(logits=torch.zeros(M, V, dtype=torch.float16)),
                dict(tokens=torch.zeros(M, dtype=torch.int64)), dict(tokens=torch.zeros(M + 1, dtype=i32)),
                dict(logprob=torch.empty(M, dtype=torch.bfloat16)), dict(rank=torch.empty(M)),
                dict(entropy=torch.empty(M - 1)), dict(topk_ids=torch.empty(M, k)),
                dict(topk_ids=torch.empty(M, 2 * k, dtype=i32)[:, ::2]), dict(topk_logprob=torch.empty(M, k + 1)),
                dict(topk_ids=None), dict(ws=torch.empty(512, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError):
            moe.moe_token_logprobs(**{**good, **bad})
    for bad in ((0, 10, 1), (1, 0, 1), (1, 10, -1)):
        with pytest.raises(ValueError):
            moe.logprobs_workspace(*bad)
    L, r, K, N = 3, 8, 32, 48
    bf = torch.bfloat16
    a, b, s = torch.zeros(L, r, K, dtype=bf), torch.zeros(L, N, r, dtype=bf), torch.ones(L)
    for bad in ((a.float(), b, s), (a, b[:2], s), (a, b.transpose(1, 2), s), (a, b[:, :, :4], s), (a, b, s[:2]),
                (a, b, s.double()), (a[0], b, s), (a, b[0], s)):
        with pytest.raises(ValueError):
            moe.lora(*bad)
    lp = moe.lora(a, b, s)
    x, ids, y = torch.zeros(M, K, dtype=bf), torch.zeros(M, dtype=i32), torch.zeros(M, N)
    good = dict(x=x, adapter_ids=ids, base=y, out=torch.empty(M, N), ws=torch.empty(4096, dtype=torch.uint8))
    for bad in (dict(x=x.float()), dict(x=torch.zeros(M, K + 1, dtype=bf)), dict(x=torch.zeros(K, M, dtype=bf).t()),
                dict(adapter_ids=ids.long()), dict(adapter_ids=ids[:2]), dict(base=y.to(bf)), dict(base=y[:2]),
                dict(out=torch.empty(M, N + 1)), dict(out=y.half()), dict(out=torch.empty(N, M).t())):
        with pytest.raises(ValueError):
            moe.moe_lora_add(lp, **{**good, **bad})
    q, w = torch.zeros(M, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    good = dict(a=q, a_scale=torch.ones(M), w=w, w_scale=torch.ones(N), lp=lp, x=x, adapter_ids=ids, out=torch.empty(M, N),
                ws=torch.empty(4096, dtype=torch.uint8))
    for bad in (dict(a=q.float()), dict(a=q[:2]), dict(a=q[:, :16]), dict(w=w[:, :16]), dict(w=w[:40]), dict(w=w.to(torch.uint8)),
                dict(a_scale=torch.ones(M + 1)), dict(w_scale=torch.ones(N).double()), dict(x=x[:2]), dict(x=x.float()),
                dict(adapter_ids=ids.long()), dict(out=torch.empty(M, N).half())):
        with pytest.raises(ValueError):
            moe.moe_int8_linear_lora(**{**good, **bad})
