"""moe_int8_linear against exact integer sums.

The sums are exact and the definition names the roundings after them
(fl32(fl32(sum) a_scale) w_scale, then bf16 where asked for), so the outputs
are compared bit for bit.
"""
import numpy as np
import pytest
import torch

from _around_gpu import Out, same_f32, up
from _around_ref import int8_product
from mxfp4_weight_streaming_amd import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _inputs(rng, M, N, K):
    a = rng.integers(-127, 128, (M, K), dtype=np.int8)
    w = rng.integers(-127, 128, (N, K), dtype=np.int8)
    return a, (0.01 + rng.random(M)).astype(np.float32), w, (0.001 + 0.01 * rng.random(N)).astype(np.float32)


def _check(moe, a, sa, w, sw, types=(torch.float32, torch.bfloat16)):
    acc, ref = int8_product(a, sa, w, sw)
    da, dsa, dw, dsw = up(a), up(sa), up(w), up(sw)
    for t in types:
        out = Out((a.shape[0], w.shape[0]), t)
        moe.moe_int8_linear(da, dsa, dw, dsw, out.t)
        torch.cuda.synchronize()
        got = out.bits()
        if t == torch.float32:
            assert same_f32(got, ref), (np.argwhere(got != ref)[:4], got[got != ref][:4], ref[got != ref][:4])
        else:
            assert np.array_equal(got, synth.bf16_from_f32(ref)), np.argwhere(got != synth.bf16_from_f32(ref))[:4]


# tokens: each GEMV bound and around, around tiles; channels and depths: one, odd, around tiles and steps
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 257])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 64), (67, 206), (130, 769), (512, 512), (259, 80)])
def test_sizes(moe, M, N, K):
    print(f"M={M} N={N} K={K}", flush=True)
    _check(moe, *_inputs(np.random.default_rng(M * 7 + N + K), M, N, K))


@pytest.mark.parametrize("M,N,K", [
    (1, 2560, 2560), (4, 1536, 2560), (8, 5003, 2560), (6, 300, 5008), (3, 33, 16), (8, 20, 70000),
    (12, 2560, 768), (77, 2563, 769), (100, 70, 4100), (200, 1000, 15), (300, 640, 2560), (512, 1536, 256),
    (513, 777, 1033), (1030, 520, 336), (2048, 256, 64), (257, 2600, 1040)])
def test_shapes(moe, M, N, K):
    print(f"M={M} N={N} K={K}", flush=True)
    _check(moe, *_inputs(np.random.default_rng(M + N + K), M, N, K))


@pytest.mark.parametrize("M", [1, 8, 16, 40, 300])
def test_largest_sums(moe, M):
    """The deepest product of the largest codes: 131071 * 128 * 128 < 2^31; and its opposite sign."""
    K, N = 131071, 40
    a = np.full((M, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1::2] = 127
    one = np.ones(M, np.float32), np.ones(N, np.float32)
    ref = np.where(np.arange(N) % 2 == 0, np.float32(131071 * 16384), np.float32(-131071 * 128 * 127))
    out = Out((M, N), torch.float32)
    moe.moe_int8_linear(up(a), up(one[0]), up(w), up(one[1]), out.t)
    torch.cuda.synchronize()
    assert same_f32(out.bits(), np.broadcast_to(ref, (M, N)))


@pytest.mark.parametrize("M", [1, 5, 20, 130])
def test_scales(moe, M):
    """Scales 0, subnormal, huge; results that overflow fp32 or bf16 are infinite."""
    rng = np.random.default_rng(20 + M)
    a, sa, w, sw = _inputs(rng, M, 70, 96)
    sw[:6] = [0.0, 1e-42, 1e30, 3e38, 1e-38, 1.0]
    sa[0] = 1e5
    with np.errstate(over="ignore", invalid="ignore"):
        acc, ref = int8_product(a, sa, w, sw)
    for t in (torch.float32, torch.bfloat16):
        out = Out((M, 70), t)
        moe.moe_int8_linear(up(a), up(sa), up(w), up(sw), out.t)
        torch.cuda.synchronize()
        want = up(ref).to(t)
        assert torch.equal(torch.nan_to_num(out.t.float()), torch.nan_to_num(want.float()))
        out.bits()


def test_long_channel_axis(moe):
    """An LM head's channel count, sampled: rows at the start, the end and between."""
    M, N, K = 12, 157184, 512
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(N, generator=g, device="cuda")
    for m in (1, 4, M):
        sa = torch.rand(m, generator=g, device="cuda")
        out = Out((m, N), torch.float32)
        moe.moe_int8_linear(a[:m], sa, w, sw, out.t)
        torch.cuda.synchronize()
        got = out.bits()
        cols = np.unique(np.concatenate([np.arange(40), np.arange(N - 40, N),
                                         np.random.default_rng(22).integers(0, N, 500)]))
        at = torch.from_numpy(cols).cuda()
        _, ref = int8_product(a[:m].cpu().numpy(), sa.cpu().numpy(), w[at].cpu().numpy(), sw[at].cpu().numpy())
        assert same_f32(got[:, cols], ref)


@pytest.mark.parametrize("M", [2, 600])
def test_output_offsets_beyond_32_bits(moe, M):
    """An output of more than 2^31 elements: its first and last rows and columns."""
    N, K = (2 ** 31 + 5000) // M, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(23)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    out = Out((M, N), torch.bfloat16)
    moe.moe_int8_linear(a, sa, w, sw, out.t)
    torch.cuda.synchronize()
    assert bool((out.raw[out.n:] == 0xA5).all())
    for cols in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
        want = (a.double() @ w[cols].double().t()).to(torch.bfloat16)
        assert torch.equal(out.t[:, cols], want)
