"""moe_add_rmsnorm and moe_int8_quantize against plain implementations in 64
bits and against the oracle's quantiser.

The definition names each rounding, and the mean square is the exact one
rounded once, so residual_out, y, codes and scales are compared bit for bit.
y is also held to the formula without roundings: fl32(r w), rstd, their product
and bf16 make |y - y64| <= |y64| (2^-8 + 3 * 2^-24 (1 + 2^-8)) < 0.00391 |y64|,
plus half the smallest bf16 number for the rounding of subnormal results.
"""
import numpy as np
import pytest
import torch

import oracle
from _around_gpu import Out, same_f32, up
from _around_ref import int8_rows, rmsnorm, widen
from mxfp4_weight_streaming_amd import synth

pytestmark = pytest.mark.gpu

F8, I8, BF, F32 = torch.float8_e4m3fn, torch.int8, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _rows(rng, M, H, bf16, size=1.0):
    v = (rng.standard_normal((M, H)) * size * np.exp(0.5 * rng.standard_normal((M, 1)))).astype(np.float32)
    return synth.bf16_from_f32(v) if bf16 else v


def _check_y(y_bits, y64):
    y = widen(y_bits).astype(np.float64)
    assert np.all(np.abs(y - y64) <= np.abs(y64) * 0.00391 + 2.0 ** -134), np.max(np.abs(y - y64) / (np.abs(y64) + 1e-300))


def _check_codes(codes, scale, y_bits, q):
    rq, rs = oracle.quant_act(y_bits) if q == F8 else int8_rows(y_bits)
    assert same_f32(scale, rs)
    assert np.array_equal(codes.view(np.uint8), rq.view(np.uint8))


def _run(moe, x, residual, weight, eps, r_bf16, q=None, want=("r", "y"), in_place=False):
    M, H = x.shape
    rt = BF if r_bf16 else F32
    res = None if residual is None else up(residual)
    ro = Out((M, H), rt) if "r" in want else None
    if in_place:
        ro.t.copy_(res)
        res = ro.t
    y = Out((M, H), BF) if "y" in want else None
    codes = Out((M, H), q) if q is not None else None
    scale = Out((M,), F32) if q is not None else None
    t = lambda o: None if o is None else o.t  # noqa: E731
    moe.moe_add_rmsnorm(up(x), res, up(weight), eps, t(ro), y=t(y), q=t(codes), scale=t(scale))
    torch.cuda.synchronize()
    return [None if o is None else o.bits() for o in (ro, y, codes, scale)]


# row lengths: one element, below and around a wave, around powers of two, odd, the layers', the largest
LENGTHS = [1, 2, 7, 8, 63, 64, 65, 255, 256, 257, 512, 520, 769, 1001, 1024, 2047, 2048, 2560, 2571, 4096, 5120, 8200,
           16384, 32760, 32767, 32768]


@pytest.mark.parametrize("H", LENGTHS)
def test_lengths(moe, H):
    rng = np.random.default_rng(1000 + H)
    M = 5 if H <= 8200 else 2
    for k, (xb, rb, wb, q) in enumerate([(False, True, True, F8), (True, False, True, I8), (True, True, False, None)]):
        x, res = _rows(rng, M, H, xb), _rows(rng, M, H, rb, 2.0)
        w = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
        w = synth.bf16_from_f32(w) if wb else w
        r, yb, y64 = rmsnorm(x, res, w, 1e-6, rb)
        ro, y, codes, scale = _run(moe, x, res, w, 1e-6, rb, q)
        print(f"H={H} types {k}", flush=True)
        assert np.array_equal(ro.view(np.uint8), r.view(np.uint8))
        _check_y(y, y64)
        assert np.array_equal(y, yb)
        if q is not None:
            _check_codes(codes, scale, yb, q)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 33, 257, 2049])
@pytest.mark.parametrize("H", [2560, 100, 64])
def test_row_counts(moe, M, H):
    rng = np.random.default_rng(2000 + M + H)
    x, res, w = _rows(rng, M, H, False), _rows(rng, M, H, True, 2.0), _rows(rng, 1, H, True)[0]
    r, yb, y64 = rmsnorm(x, res, w, 1e-5, True)
    ro, y, codes, scale = _run(moe, x, res, w, 1e-5, True, F8)
    assert np.array_equal(ro, r) and np.array_equal(y, yb)
    _check_y(y, y64)
    _check_codes(codes, scale, yb, F8)


@pytest.mark.parametrize("q", [F8, I8, torch.uint8])
def test_each_output_alone(moe, q):
    """Outputs that are not asked for change nothing; uint8 codes are E4M3 codes."""
    rng = np.random.default_rng(3)
    H, M = 264, 6
    x, res, w = _rows(rng, M, H, True), _rows(rng, M, H, True), _rows(rng, 1, H, False)[0]
    r, yb, _ = rmsnorm(x, res, w, 1e-6, True)
    assert np.array_equal(_run(moe, x, res, w, 1e-6, True, None, ("r",))[0], r)
    assert np.array_equal(_run(moe, x, res, w, 1e-6, True, None, ("y",))[1], yb)
    _, _, codes, scale = _run(moe, x, res, w, 1e-6, True, q, ())
    _check_codes(codes, scale, yb, F8 if q == torch.uint8 else q)


@pytest.mark.parametrize("bf16", [True, False])
def test_no_residual(moe, bf16):
    rng = np.random.default_rng(4)
    x, w = _rows(rng, 3, 640, False), _rows(rng, 1, 640, True)[0]
    r, yb, _ = rmsnorm(x, None, w, 1e-6, bf16)
    ro, y, _, _ = _run(moe, x, None, w, 1e-6, bf16)
    assert np.array_equal(ro.view(np.uint8), r.view(np.uint8)) and np.array_equal(y, yb)
    # without residual_out either, r keeps x's type
    y2 = _run(moe, x, None, w, 1e-6, False, None, ("y",))[1]
    assert np.array_equal(y2, rmsnorm(x, None, w, 1e-6, False)[1])


@pytest.mark.parametrize("H", [2560, 1001])
@pytest.mark.parametrize("bf16", [True, False])
def test_in_place_residual(moe, H, bf16):
    rng = np.random.default_rng(5 + H)
    x, res, w = _rows(rng, 70, H, False), _rows(rng, 70, H, bf16), _rows(rng, 1, H, True)[0]
    r, yb, _ = rmsnorm(x, res, w, 1e-6, bf16)
    ro, y, codes, scale = _run(moe, x, res, w, 1e-6, bf16, I8, in_place=True)
    assert np.array_equal(ro.view(np.uint8), r.view(np.uint8)) and np.array_equal(y, yb)
    _check_codes(codes, scale, yb, I8)


@pytest.mark.parametrize("q", [F8, I8])
@pytest.mark.parametrize("H", [2560, 333])
def test_extreme_rows(moe, q, H):
    """Rows of zeros, of one value, with one huge or only tiny values, and rows that cancel to zero."""
    rng = np.random.default_rng(6)
    x = np.zeros((9, H), np.float32)
    x[1] = 3.0
    x[2, H // 2] = -1e15
    x[3] = 1e-30 * rng.standard_normal(H)          # rstd = 1 / sqrt(eps): y far below 2^-64 with w 1e-3
    x[4] = 1e18 * rng.standard_normal(H)           # squares beyond fp32
    x[5] = rng.standard_normal(H)
    x[6] = 1e-40                                   # subnormal
    x[7] = rng.standard_normal(H)
    x[8, 0] = 1.0
    res = np.zeros((9, H), np.float32)
    res[5] = -x[5]
    for w in (np.ones(H, np.float32), np.full(H, 1e-3, np.float32), np.zeros(H, np.float32)):
        r, yb, _ = rmsnorm(x, res, w, 1e-6, False)
        ro, y, codes, scale = _run(moe, x, res, w, 1e-6, False, q)
        assert same_f32(ro, r) and np.array_equal(y, yb)
        _check_codes(codes, scale, yb, q)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (301, 512), (4, 2560), (70, 2571), (2, 70001)])
def test_int8_quantize(moe, rows, cols):
    rng = np.random.default_rng(7 + cols)
    v = _rows(rng, rows, cols, True)
    v[0] = 0
    if rows > 2:
        v[1] = synth.bf16_from_f32(np.full(cols, -2e38, np.float32))
        v[2] = synth.bf16_from_f32((1e-25 * rng.standard_normal(cols)).astype(np.float32))   # amax < 2^-64
    q, s = Out((rows, cols), I8), Out((rows,), F32)
    moe.moe_int8_quantize(up(v), q.t, s.t)
    torch.cuda.synchronize()
    _check_codes(q.bits(), s.bits(), v, I8)


def test_matches_quant_act(moe):
    """The E4M3 codes are those moe_quant_act gives for y, which moe_experts_forward takes."""
    rng = np.random.default_rng(8)
    M, H = 4, 2560
    x, res, w = _rows(rng, M, H, False), _rows(rng, M, H, True), _rows(rng, 1, H, True)[0]
    y, q, s = Out((M, H), BF), Out((M, H), F8), Out((M,), F32)
    moe.moe_add_rmsnorm(up(x), up(res), up(w), 1e-6, None, y=y.t, q=q.t, scale=s.t)
    q2, s2 = Out((M, H), torch.uint8), Out((M,), F32)
    moe.moe_quant_act(moe.shape(H, 768, 256, 8), M, y.t, q2.t, s2.t)
    torch.cuda.synchronize()
    assert np.array_equal(q.bits(), q2.bits()) and same_f32(s.bits(), s2.bits())
