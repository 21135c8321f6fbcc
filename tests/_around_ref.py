"""Plain implementations, on the host in 64 bits, of the operators around the
expert layer, and of the roundings their definitions name."""
from __future__ import annotations

import math

import numpy as np

from mxfp4_weight_streaming_amd import synth

f32, f64 = np.float32, np.float64


def widen(a: np.ndarray) -> np.ndarray:
    """bf16 bits (uint16) or float32 as float32."""
    return synth.bf16_to_f32(a) if a.dtype == np.uint16 else a


def stored(r: np.ndarray, bf16: bool) -> np.ndarray:
    """A float32 row as it is stored: itself, or its bf16 bits."""
    return synth.bf16_from_f32(r) if bf16 else r


def rmsnorm(x, residual, weight, eps: float, bf16: bool):
    """(r as stored, y bits, y in 64 bits without the roundings after r) of rows x [M,H]."""
    r = widen(x)
    if residual is not None:
        r = widen(residual) + r
    r = stored(r, bf16)
    rf, w = widen(r), widen(weight)
    H = rf.shape[1]
    # the exact sum of squares, rounded once
    ss = np.array([math.fsum(v) for v in (rf.astype(f64) ** 2)])
    rstd = 1.0 / np.sqrt(ss / H + eps)
    y = ((rf * w) * rstd.astype(f32)[:, None]).astype(f32)
    return r, synth.bf16_from_f32(y), rf.astype(f64) * w.astype(f64) * rstd[:, None]


def int8_rows(y_bits):
    """(codes, scales) of bf16 rows: s = amax / 127, codes of the rounded quotient, to nearest even."""
    y = widen(y_bits)
    amax = np.abs(y).max(axis=1)
    s = np.where(amax == 0, f32(1), amax / f32(127)).astype(f32)
    return np.rint(y / s[:, None]).astype(np.int8), s


def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """fp64 scores of one token's logits; -inf and NaN score 0."""
    x = logits.astype(f64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(f32).max))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    if not np.isfinite(x).any():
        return np.zeros_like(x)
    e = np.exp(x - x.max())
    return e / math.fsum(e)


def route(logits, bias, K, score, groups=1, group_topk=1, group_score=2, renormalise=True, factor=1.0):
    """(ids [M,K], w [M,K] float64) by sorting, token by token."""
    M, E = logits.shape
    each = E // groups
    ids = np.zeros((M, K), np.int32)
    w = np.zeros((M, K), f64)
    for m in range(M):
        s = scores(logits[m], score).astype(f32)      # rounded: a score below fp32's range is 0
        c = s if bias is None else s + bias
        there = ~(np.isnan(logits[m]) | np.isneginf(logits[m]) | np.isnan(c) | np.isneginf(c))
        value = []
        for g in range(groups):
            mine = sorted((c[e] for e in range(g * each, (g + 1) * each) if there[e]), reverse=True)[:group_score]
            v = f32(-np.inf)
            if mine:
                v = mine[0]
                for more in mine[1:]:
                    v = f32(v + more)
            value.append(v)
        kept = sorted(range(groups), key=lambda g: (-float(value[g]), g))[:group_topk]
        cand = [e for g in kept for e in range(g * each, (g + 1) * each)]
        cand.sort(key=lambda e: (not there[e], -float(c[e]) if there[e] else 0.0, e))
        ids[m] = cand[:K]
        v = np.where(there[ids[m]], s[ids[m]].astype(f64), 0.0)
        if renormalise and v.sum() != 0.0:
            v = v / v.sum()
        w[m] = v * factor
    return ids, w


def int8_product(a, a_scale, w, w_scale):
    """(exact int64 sums, the fp32 result of the definition's roundings)."""
    acc = a.astype(np.int64) @ w.astype(np.int64).T
    return acc, (acc.astype(f32) * a_scale.astype(f32)[:, None]) * w_scale.astype(f32)[None, :]
