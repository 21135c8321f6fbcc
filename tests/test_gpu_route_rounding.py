"""The rounding of moe_route_scores' scores: fp64 evaluations, rounded once.

With as many experts as K, no bias, no renormalisation and a factor of 1 the
weights are the scores.  Of two experts with logits a > b, softmax gives the
second 1 / (1 + e^(a - b)); a - b is exact in fp64, so the kernel's evaluation
is off by at most 2^-51.8 (exponential) + 2^-53 (the sum 1 + e) + 2^-52 (the
reciprocal) + 2^-53 (the product) < 2^-50 of it, sigmoid's by less: the score is
the correctly rounded one wherever the exact one is farther than that from the
middle between two fp32 numbers.
"""
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest
import torch

from _around_gpu import Out, up

pytestmark = pytest.mark.gpu

# Pairs of logits whose second score lies between 2^-50 and 2^-46 of itself from
# the middle between two fp32 numbers, where an exponential off by 2^-46 falls
# on the other side.
NEAR_MIDDLE = [
    ("0x1.152102p+3", "-0x1.e0cf8ep-9"), ("0x1.1543b4p+3", "-0x1.24a97p-9"), ("0x1.154fc2p+3", "-0x1.8f25cp-11"),
    ("0x1.1fb574p+2", "-0x1.8dffeep-9"), ("0x1.2265cp+2", "-0x1.159f24p-9"), ("0x1.31c56p+1", "-0x1.c7e72ap-9"),
    ("0x1.427bd8p+3", "-0x1.415048p-9"), ("0x1.428876p+3", "-0x1.ddc12p-11"), ("0x1.4de1b4p+2", "-0x1.f10bdp-11"),
    ("0x1.578742p+3", "-0x1.c9b4dp-12"), ("0x1.6cdddep+3", "-0x1.04c404p-10"), ("0x1.6ce418p+3", "-0x1.9bd58ap-9"),
    ("0x1.6dd98cp+3", "-0x1.a947dap-9"), ("0x1.775564p+2", "-0x1.f68908p-11"), ("0x1.7a9a2cp+2", "-0x1.cc3cc8p-11"),
    ("0x1.831be4p+3", "-0x1.9e195p-9"), ("0x1.831eeep+3", "-0x1.6d795p-9"), ("0x1.83da26p+3", "-0x1.f3e39p-11"),
    ("0x1.99409p+3", "-0x1.3550eap-9"), ("0x1.b05bb6p+3", "-0x1.90bd28p-11"), ("0x1.b6464p+0", "-0x1.f3d064p-10"),
    ("0x1.d0c2dp+2", "-0x1.d2dc1p-12"), ("0x1.d338a8p+2", "-0x1.74289p-12"), ("0x1.dc65bap+3", "-0x1.ea2a4p-10"),
    ("0x1.e6e3fp+1", "-0x1.aafe8p-10"), ("0x1.f1f27ep+3", "-0x1.a2c23p-9"), ("0x1.f25e9cp+3", "-0x1.8f617cp-9"),
    ("0x1.f3378p+3", "-0x1.abaeccp-9"), ("0x1.f36142p+3", "-0x1.dfaea4p-10"),
]


@pytest.fixture(scope="module")
def moe():
    from mxfp4_weight_streaming_amd import binding
    return binding


def _scores(moe, logits, score):
    """The scores of logits [M,E], E <= 8, in the experts' order."""
    M, E = logits.shape
    ids, w = Out((M, E), torch.int32), Out((M, E), torch.float32)
    moe.moe_route_scores(moe.router(E, E, score=score, renormalise=False), up(logits), None, ids.t, w.t)
    torch.cuda.synchronize()
    s = np.empty((M, E), np.float32)
    np.put_along_axis(s, ids.bits().astype(np.int64), w.bits(), 1)
    return s


def _rounded(exact: Decimal) -> np.float32:
    """The fp32 number next to a positive number given to many digits."""
    f = np.float32(float(exact))
    around = (np.nextafter(f, np.float32(0)), f, np.nextafter(f, np.float32(np.inf)))
    return min(around, key=lambda v: abs(Fraction(float(v)) - Fraction(exact)))


def test_softmax_near_the_middle(moe):
    getcontext().prec = 50
    logits = np.array([[float.fromhex(a), float.fromhex(b)] for a, b in NEAR_MIDDLE], np.float32)
    assert np.array_equal(logits.astype(np.float64), [[float.fromhex(v) for v in p] for p in NEAR_MIDDLE])
    want = []
    for a, b in logits.astype(np.float64):
        e = (Decimal(b) - Decimal(a)).exp()
        want.append(_rounded(e / (1 + e)))
    got = _scores(moe, logits, "softmax")[:, 1]
    assert got.tolist() == [float(v) for v in want]


def test_sigmoid_scores(moe):
    """Four million scores of logits from 2^-8 to 104 against long double ones, rounded to fp32."""
    rng = np.random.default_rng(16)
    mag = np.exp2(rng.uniform(-8.0, np.log2(104.0), (1 << 19, 8)))
    logits = (mag * rng.choice([-1.0, 1.0], mag.shape)).astype(np.float32)
    exact = 1 / (1 + np.exp(-logits.astype(np.longdouble)))
    want = exact.astype(np.float32)
    got = _scores(moe, logits, "sigmoid")
    off = np.nonzero(got != want)
    for g, w, x in zip(got[off], want[off], exact[off]):
        middle = (np.longdouble(g) + np.longdouble(w)) / 2       # the exact score lies next to it
        assert abs(x / middle - 1) < 2.0 ** -50 and abs(int(g.view(np.int32)) - int(w.view(np.int32))) == 1, (g, w)
