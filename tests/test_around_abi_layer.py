"""CPU-only checks of moe_decode_forward_scored's refusals: outputs and
workspace that share bytes with an input or with each other, and the status of
each bad router."""
import ctypes

import pytest

FAR = 1 << 40        # addresses that share no byte, never dereferenced: validation fails first
H, I, E, K, M = 2560, 768, 64, 8, 4
NAMES = ["hidden", "router_w", "bias", "w13", "w13_scale", "w2", "w2_scale", "sh_w13", "sh_w13_scale", "sh_w2",
         "sh_w2_scale", "out", "ws"]
SIZE = dict(hidden=M * H * 2, router_w=E * H * 2, bias=E * 4, w13=E * I * H, w13_scale=E * 2 * I * H // 32,
            w2=E * H * I // 2, w2_scale=E * H * I // 32, sh_w13=I * H, sh_w13_scale=2 * I * H // 32, sh_w2=H * I // 2,
            sh_w2_scale=H * I // 32, out=M * H * 4)
INPUTS = NAMES[:-2]


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _call(moe, at=None, router=None, ws_bytes=None, tokens=M, **change):
    """The call on distinct addresses but for `at`; its status."""
    p = {n: FAR * (i + 1) for i, n in enumerate(NAMES)}
    p.update(at or {})
    shp = moe.shape(H, I, E, K)
    rp = moe.router(E, K, score="sigmoid", groups=4, group_topk=2)
    for k, v in (router or {}).items():
        setattr(rp, k, v)
    sh = moe.MoeSharedExpert(p["sh_w13"], p["sh_w13_scale"], p["sh_w2"], p["sh_w2_scale"])
    n = moe.moe_workspace_bytes(shp, tokens) if ws_bytes is None else ws_bytes
    return moe.raw().moe_decode_forward_scored(
        ctypes.byref(shp), ctypes.byref(rp), tokens, p["hidden"], p["router_w"], p["bias"], p["w13"], p["w13_scale"],
        p["w2"], p["w2_scale"], ctypes.byref(sh), p["out"], p["ws"], n, None)


@pytest.mark.parametrize("name", INPUTS)
def test_output_over_an_input(moe, name):
    base = FAR * (NAMES.index(name) + 1)
    end = base + SIZE[name]
    last = end - 1 - (end - 1) % 16                      # the last aligned address inside the input
    for at in (dict(out=base), dict(out=last), dict(ws=base), dict(ws=end - 1 - (end - 1) % 256)):
        assert _call(moe, at) == -1
        assert "overlaps" in moe.moe_last_error() and name.removeprefix("sh_") in moe.moe_last_error()
    # the input's first byte is the last of out, or of the workspace's used part
    need = moe.moe_workspace_bytes(moe.shape(H, I, E, K), M)
    assert _call(moe, dict(out=base + 16 - SIZE["out"])) == -1
    assert _call(moe, dict(ws=base + 256 - need)) == -1


def test_out_over_the_workspace(moe):
    base = FAR * (NAMES.index("ws") + 1)
    need = moe.moe_workspace_bytes(moe.shape(H, I, E, K), M)
    for at in (base, base + need - 256, base - SIZE["out"] + 16):
        assert _call(moe, dict(out=at)) == -1
        assert "the workspace overlaps out" in moe.moe_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(num_experts=0), -1), (dict(topk=0), -1), (dict(num_groups=5), -1), (dict(score=2), -1),
    (dict(group_topk=5), -1), (dict(group_score=3), -1), (dict(factor=float("nan")), -1),
    (dict(num_groups=16, group_topk=1), -1),
    (dict(num_experts=1024), -2), (dict(topk=9), -2), (dict(num_experts=512, num_groups=128, group_topk=8), -2)])
def test_status_of_a_bad_router(moe, change, status):
    assert _call(moe, router=change) == status
