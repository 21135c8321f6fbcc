"""Plain implementations, in 64 bits on the host, of the log probabilities and
the adapters, and how far the library's fp32 arithmetic may be from them."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24                   # half a step of fp32, relative
F32_MAX = float(torch.finfo(torch.float32).max)


def clean(logits: torch.Tensor) -> torch.Tensor:
    """A row of logits as the definitions count it, in 64 bits: NaN is -inf, +inf the largest finite fp32 value."""
    x = logits.detach().cpu().double()
    return torch.where(torch.isnan(x), -torch.inf, x).clamp(max=F32_MAX)


class Logprobs:
    """What moe_token_logprobs gives for `logits` [M,V] and `tokens` [M], and bounds of its errors.

    The sums are over d = l - max, without the largest's own term.  Off by rounding are, relative to a term e^d: d itself
    and its product by log2(e) (2.2 U |d|), the exponential (2 U), and the sum of a term's group (at most 16 terms in fp32,
    in turn: 16 U; longer sums are kept in 64 bits).  So S - 1 is off by at most sum e^d (2.5 |d| + 24) U, T by
    sum e^d |d| (2.5 |d| + 26) U, and each output by half a step more."""

    def __init__(self, logits, tokens, k):
        x = clean(logits)
        M, V = x.shape
        t = tokens.cpu().long()
        top, where = x.max(1, keepdim=True)
        empty = top[:, 0] == -torch.inf
        d = torch.where(torch.isinf(x), -torch.inf, x - torch.where(empty[:, None], 0.0, top))
        e = torch.exp(d)
        e1 = e.scatter(1, where, 0.0)
        fin = torch.where(e1 > 0, d, 0.0)
        s1 = e1.sum(1)
        s_err = (e1 * (2.5 * fin.abs() + 24)).sum(1) * U
        t_sum, t_err = (e1 * fin).sum(1), (e1 * fin.abs() * (2.5 * fin.abs() + 26)).sum(1) * U
        S = 1 + s1
        log_s = torch.log1p(s1)
        log_err = s_err / S
        self.entropy = torch.where(empty, 0.0, log_s - t_sum / S)
        self.entropy_err = log_err + t_err / S + t_sum.abs() / S * log_err + U * self.entropy + 1e-38
        logp = torch.where(d == -torch.inf, -torch.inf, d - log_s[:, None])
        asked = t.clamp(0, V - 1)[:, None]
        mine, lp = x.gather(1, asked), logp.gather(1, asked)[:, 0]
        i = torch.arange(V)
        rank = ((x > mine) | ((x == mine) & (i < asked))).sum(1)
        self.logprob = torch.where(t < 0, 0.0, torch.where(t >= V, -torch.inf, lp))
        self.rank = torch.where(t < 0, -1, torch.where(t >= V, V, rank))
        self.log_err = log_err
        order = torch.sort(x, dim=1, descending=True, stable=True)
        n = min(k, V)
        ids, vals = order.indices[:, :n], logp.gather(1, order.indices[:, :n])
        ids = torch.where(vals == -torch.inf, -1, ids)
        self.ids = torch.nn.functional.pad(ids, (0, k - n), value=-1)
        self.top = torch.nn.functional.pad(vals, (0, k - n), value=-torch.inf)

    def check(self, logprob=None, rank=None, entropy=None, ids=None, top=None):
        for got, ref, err in ((logprob, self.logprob, self.log_err), (top, self.top, self.log_err[:, None])):
            if got is None:
                continue
            got = torch.as_tensor(np.asarray(got)).double()
            fin = torch.isfinite(ref)
            # (a value beyond fp32's range is -inf there)
            fin &= ref >= -F32_MAX
            assert bool((got[~fin] == -torch.inf).all()), (got[~fin], ref[~fin])
            far = (got - ref).abs() - (err + U * ref.abs() + 1e-38)
            assert bool((far[fin] <= 0).all()), (float(far[fin].max()), torch.nonzero(far * fin > 0)[:4])
        if entropy is not None:
            got = torch.as_tensor(np.asarray(entropy)).double()
            far = (got - self.entropy).abs() - self.entropy_err
            assert bool((far <= 0).all()), (float(far.max()), torch.nonzero(far > 0)[:4])
        if rank is not None:
            assert np.array_equal(np.asarray(rank), self.rank.numpy()), (rank, self.rank)
        if ids is not None:
            assert np.array_equal(np.asarray(ids), self.ids.numpy()), np.argwhere(np.asarray(ids) != self.ids.numpy())[:4]


def lora_delta(x, a, b, scale, ids):
    """B (scale A x) of each row in 64 bits, and how far fp32 sums may be from it.

    A sum of n products of bf16 values is exact but for the roundings of its partial sums: a chain of at most n / 16 + 40
    of them in any of the kernels (64 lanes or 4 waves share the n terms, 16 or more at a time), each at most a step (2 U)
    of the sum of magnitudes."""
    x, a, b = (t.detach().cpu().double() for t in (x, a, b))
    L, r, K = a.shape
    M, N = x.shape[0], b.shape[1]
    ids = ids.cpu().long()
    d, err = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for i in torch.unique(ids).tolist():
        if i < 0 or i >= L:
            continue
        rows = torch.nonzero(ids == i)[:, 0]
        s = 1.0 if scale is None else float(scale[i])
        u, mag = s * (x[rows] @ a[i].t()), abs(s) * (x[rows].abs() @ a[i].abs().t())
        d[rows] = u @ b[i].t()
        u_err = 2 * U * (K / 16 + 40) * mag + 2 * U * u.abs()
        err[rows] = u_err @ b[i].abs().t() + 2 * U * (r / 16 + 40) * (u.abs() @ b[i].abs().t())
    return d, err


def check_rows(got, ref, err, dtype):
    """got = the reference rounded to its type, off by err and fp32's last additions before that."""
    got = torch.as_tensor(np.asarray(got)).double() if not isinstance(got, torch.Tensor) else got.detach().cpu().double()
    half = torch.finfo(dtype).eps / 2
    far = (got - ref).abs() - (err + 4 * U * ref.abs() + half * (ref.abs() + err) + 1e-38)
    assert bool((far <= 0).all()), (float(far.max()), torch.nonzero(far > 0)[:4], got[far > 0][:4], ref[far > 0][:4])
