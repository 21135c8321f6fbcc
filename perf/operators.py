"""Measured cases of the operators around the expert layer: the residual add with
RMS norm and 8-bit output, the routing by scores, and the int8 matrix product.

``run`` computes each operator in its plain form (elementary torch operations),
or, where ``own`` is true, by the library's calls.

The definitions, which both sides follow:

* norm: r = residual + x, rounded to the residual's type; rstd = 1/sqrt(mean(r^2) + eps)
  in 64 bits, rounded to fp32; y = bf16((r w) rstd) with both products rounded to fp32;
  8-bit codes of y with one scale a token, s = amax/448 (E4M3) or amax/127 (int8),
  1 for a row of zeros, codes of the correctly rounded quotient y/s.
* routing: scores s = sigmoid or softmax of the logits, evaluated in 64 bits and rounded
  to fp32; choice values c = s + bias in fp32.  An expert whose logit is -inf or NaN, or
  whose c is -inf or NaN, is unavailable.  A group's value is the sum of its n largest
  available c; the group_topk best groups stay, and of their experts the K largest c are
  taken (unavailable ones last), ties to the lowest index.  Weights: s of the taken experts,
  0 for unavailable ones, divided by their sum where they are renormalised, times a factor.
* int8 product: out[m,n] = a_scale[m] w_scale[n] sum_k a[m,k] w[n,k].
"""
import math

import torch

own = False

DEVICE = "cuda"
F32_MAX = torch.finfo(torch.float32).max
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases --------------------------------------------------------------
def _norm(tokens, hidden, x, residual, q, name=None):
    return _named(name, op="norm", tokens=tokens, hidden=hidden, x=x, residual=residual, q=q)


def _route(tokens, experts, topk, score, groups, group_topk, bias, masked=0.0, renorm=True, factor=2.5, name=None):
    return _named(name, op="route", tokens=tokens, experts=experts, topk=topk, score=score, groups=groups,
                  group_topk=group_topk, bias=bias, masked=masked, renorm=renorm, factor=factor)


def _int8(tokens, channels, depth, out, name=None):
    return _named(name, op="int8", tokens=tokens, channels=channels, depth=depth, out=out)


def _named(name, **case):
    return case if name is None else dict(case, name=name)


def listed():
    return [
        # one decode token between two expert layers: the layer's fp32 output added to the bf16 residual
        _norm(1, 2560, "f32", "bf16", "e4m3", name="norm_decode_1"),
        # a prefill chunk ahead of the int8 projections
        _norm(512, 2560, "f32", "bf16", "int8", name="norm_chunk_512"),
        # the norm of a narrow, odd-sized latent row, fp32 residual, no 8-bit output
        _norm(301, 1001, "bf16", "f32", "none", name="norm_odd_1001"),
        # a long prompt in one call
        _norm(16384, 2560, "f32", "bf16", "e4m3", name="norm_prompt_16384"),
        # one decode token over all 512 experts: sigmoid scores, balance bias, 4 of 8 groups
        _route(1, 512, 8, "sigmoid", 8, 4, True, name="route_decode_1"),
        # a prefill chunk with softmax scores over 256 experts, no groups
        _route(512, 256, 8, "softmax", 1, 1, False, factor=1.0, name="route_chunk_512"),
        # a long prompt over 512 experts
        _route(16384, 512, 8, "sigmoid", 8, 4, True, name="route_prompt_16384"),
        # a dense projection for one decode token
        _int8(1, 2560, 2560, "bf16", name="int8_decode_1"),
        # the LM head over a 4-token verify window
        _int8(4, 157184, 2560, "f32", name="int8_head_4"),
        # a ragged batch: no size a multiple of a tile, rows that start at odd addresses
        _int8(77, 2563, 769, "bf16", name="int8_ragged_77"),
        # a dense projection of a long chunk
        _int8(2048, 2560, 2560, "bf16", name="int8_chunk_2048"),
        # the LM head over every position of a prefill chunk
        _int8(512, 157184, 2560, "f32", name="int8_head_512"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _rough(rng, lo, hi):
    """As _log; half of them are made multiples of 64 where they are large enough."""
    n = _log(rng, lo, hi)
    return n // 64 * 64 if n >= 128 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "route", "int8"])
    if op == "norm":
        hidden = _rough(rng, 32, 8192)
        tokens = min(_log(rng, 1, 16384), 16384 * 2560 // hidden)
        return _norm(tokens, hidden, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]),
                     rng.choice(["e4m3", "int8", "none"]))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        size = _log(rng, max(1, 8 // groups), 512 // groups)
        group_topk = rng.randint(1, groups)
        topk = min(rng.randint(1, 8), group_topk * size)
        return _route(_log(rng, 1, 16384), groups * size, topk, rng.choice(["sigmoid", "softmax"]), groups, group_topk,
                      rng.random() < 0.7, rng.choice([0.0, 0.0, 0.3]), rng.random() < 0.8, rng.choice([1.0, 2.5]))
    depth = _rough(rng, 16, 8192)
    channels = _rough(rng, 16, 157184 * 2560 // max(depth, 2560))
    most = min(512 * 157184 * 2560 // (channels * depth), 512 * 157184 // channels)
    return _int8(min(_log(rng, 1, 4096), most), channels, depth, rng.choice(["bf16", "f32"]))


# ---- inputs -------------------------------------------------------------------
def _rows_to_int8(x):
    """Row-wise int8 codes and scales of a matrix, as a loader makes them."""
    s = x.abs().amax(1) / 127.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.round(x / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEVICE)  # noqa: E731
    uniform = lambda *shape: torch.rand(shape, generator=g, device=DEVICE)  # noqa: E731
    empty = lambda shape, t: torch.empty(shape, dtype=t, device=DEVICE)  # noqa: E731
    st = dict(case)
    M = case["tokens"]
    if case["op"] == "norm":
        H = case["hidden"]
        # tokens differ in size, and a few channels carry much larger values than the rest
        size = torch.exp(0.5 * normal(M, 1)) * torch.where(uniform(1, H) < 0.01, 20.0, 1.0)
        st["x"] = (normal(M, H) * size).to(TYPES[case["x"]])
        st["residual"] = (normal(M, H) * size * 2.0).to(TYPES[case["residual"]])
        st["weight"] = (1.0 + 0.2 * normal(H)).to(torch.bfloat16)
        st["eps"] = 1e-6
        st["residual_out"], st["y"] = empty((M, H), TYPES[case["residual"]]), empty((M, H), torch.bfloat16)
        st["codes"] = {"e4m3": empty((M, H), torch.float8_e4m3fn), "int8": empty((M, H), torch.int8), "none": None}[case["q"]]
        st["scale"] = None if case["q"] == "none" else empty((M,), torch.float32)
    elif case["op"] == "route":
        E, K = case["experts"], case["topk"]
        st["logits"] = normal(M, E)
        if case["masked"] > 0.0:  # experts that are not to be had for a token; now and then none is left
            gone = uniform(M, E) < case["masked"]
            gone |= uniform(M, 1) < 0.02
            st["logits"] = st["logits"].masked_fill(gone, float("-inf"))
        st["bias"] = 0.1 * normal(E) if case["bias"] else None
        st["topk_ids"], st["topk_w"] = empty((M, K), torch.int32), empty((M, K), torch.float32)
    else:
        N, K = case["channels"], case["depth"]
        st["a"], st["a_scale"] = _rows_to_int8(normal(M, K) * torch.exp(0.3 * normal(M, 1)))
        st["w"], st["w_scale"] = _rows_to_int8(0.02 * normal(N, K))
        st["out"] = empty((M, N), TYPES[case["out"]])
    return st


# ---- one pass -------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    return {"norm": _plain_norm, "route": _plain_route, "int8": _plain_int8}[st["op"]](st)


def _run_own(st):
    from mxfp4_weight_streaming_amd import binding as moe
    if st["op"] == "norm":
        moe.moe_add_rmsnorm(st["x"], st["residual"], st["weight"], st["eps"], st["residual_out"], y=st["y"],
                            q=st["codes"], scale=st["scale"])
        return st["residual_out"], st["y"], st["codes"], st["scale"]
    if st["op"] == "route":
        if "router" not in st:  # a program makes the description of its router once
            st["router"] = moe.router(st["experts"], st["topk"], score=st["score"], groups=st["groups"],
                                      group_topk=st["group_topk"], group_score=2, renormalise=st["renorm"],
                                      factor=st["factor"])
        moe.moe_route_scores(st["router"], st["logits"], st["bias"], st["topk_ids"], st["topk_w"])
        return st["topk_ids"], st["topk_w"]
    moe.moe_int8_linear(st["a"], st["a_scale"], st["w"], st["w_scale"], st["out"])
    return st["out"]


def _plain_norm(st):
    r = (st["residual"].float() + st["x"].float()).to(st["residual"].dtype)
    # the mean square in 64 bits: 8-bit codes and scales hang on which side of a border y falls
    rstd = (1.0 / torch.sqrt(r.double().square().mean(1, keepdim=True) + st["eps"])).float()
    y = ((r.float() * st["weight"].float()) * rstd).to(torch.bfloat16)
    if st["q"] == "none":
        return r, y, None, None
    amax = y.float().abs().amax(1)
    # by a division of two tensors: torch divides by a number through its reciprocal
    s = amax / torch.full_like(amax, 448.0 if st["q"] == "e4m3" else 127.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    codes = y.float() / s[:, None]
    return r, y, codes.to(torch.float8_e4m3fn) if st["q"] == "e4m3" else torch.round(codes).to(torch.int8), s


def _plain_route(st):
    M, E = st["logits"].shape
    G, K = st["groups"], st["topk"]
    # scores in 64 bits, rounded once: experts whose values are next to each other have to keep their order
    x = st["logits"].double()
    x = torch.where(torch.isnan(x), float("-inf"), x).clamp(max=F32_MAX)
    if st["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        total = e.sum(1, keepdim=True)
        s = e / torch.where(total == 0, 1.0, total)
    s = s.float()
    c = s if st["bias"] is None else s + st["bias"]
    gone = torch.isinf(x) | torch.isnan(c) | (c == float("-inf"))
    c = torch.where(gone, float("-inf"), c)
    n = min(2, E // G)
    best = torch.sort(c.view(M, G, E // G), dim=2, descending=True, stable=True).values[:, :, :n]
    value = torch.where(torch.isinf(best), 0.0, best).sum(2)
    value = torch.where(best[:, :, 0] == float("-inf"), float("-inf"), value)
    kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, : st["group_topk"]]
    out = torch.ones((M, G), dtype=torch.uint8, device=c.device).scatter_(1, kept, 0)
    out = out.repeat_interleave(E // G, dim=1)
    order = torch.sort(c, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(out.gather(1, order), dim=1, stable=True).indices)
    ids = order[:, :K]
    w = torch.where(gone, 0.0, s).gather(1, ids)
    if st["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return ids.to(torch.int32), w * st["factor"]


def _plain_int8(st):
    acc = st["a"].float() @ st["w"].float().t()
    return (acc * st["a_scale"][:, None] * st["w_scale"]).to(st["out"].dtype)


# ---- the definitions in 64 bits ----------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "int8": _exact_int8}[case["op"]](st)


def _exact_norm(st):
    H = st["hidden"]
    r = torch.add(st["x"].double(), st["residual"].double())
    # two fp32 (or bf16) numbers' sum, as it is stored
    r = r.to(torch.float32).to(st["residual"].dtype).double()
    w = st["weight"].double()
    rstd = torch.rsqrt((r * r).sum(1) / H + st["eps"])
    y = torch.einsum("mh,h,m->mh", r, w, rstd)
    if st["q"] == "none":
        return r, y, None, None
    # what is quantised is the stored bf16 row, so its roundings belong to the scale's definition
    rounded = (r * w).to(torch.float32).double() * rstd.to(torch.float32).double()[:, None]
    rounded = rounded.to(torch.float32).to(torch.bfloat16).double()
    top = rounded.abs().max(1).values
    s = torch.where(top > 0, top / (448.0 if st["q"] == "e4m3" else 127.0), torch.ones_like(top))
    return r, y, rounded / s[:, None] if st["q"] == "e4m3" else None, s


def _exact_route(st):
    M, E = st["logits"].shape
    G, K, each = st["groups"], st["topk"], st["experts"] // st["groups"]
    weights = torch.zeros((M, K), dtype=torch.float64, device=st["logits"].device)
    index = torch.arange(E, device=st["logits"].device)
    for at in range(0, M, 512):
        x = st["logits"][at:at + 512].double()
        if st["score"] == "sigmoid":
            s = torch.sigmoid(x)
        else:
            s = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        c = s.to(torch.float32) + (0.0 if st["bias"] is None else st["bias"])
        there = torch.isfinite(x)
        low = torch.finfo(torch.float32).min
        c = torch.where(there, c, low)
        # an expert's place: how many are better, or as good and before it
        def places(v):
            n = v.shape[1]
            i = torch.arange(n, device=v.device)
            better = v[:, None, :] > v[:, :, None]
            same = (v[:, None, :] == v[:, :, None]) & (i[None, None, :] < i[None, :, None])
            return (better | same).sum(2)
        inside = places(c.reshape(-1, each)).reshape(-1, E)
        counted = torch.where((inside < 2) & there, c, torch.zeros_like(c)).reshape(-1, G, each).sum(2)
        counted = torch.where(there.reshape(-1, G, each).any(2), counted, low)
        stays = (places(counted) < st["group_topk"]).repeat_interleave(each, 1)
        place = places(torch.where(stays, c.double(), 2.0 * low))
        ids = torch.zeros((x.shape[0], K), dtype=torch.int64, device=x.device)
        row, col = torch.nonzero(place < K, as_tuple=True)
        ids[row, place[row, col]] = index[col]
        w = torch.where(there, s, torch.zeros_like(s)).gather(1, ids)
        if st["renorm"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
        weights[at:at + 512] = w * st["factor"]
    return None, weights


def _exact_int8(st):
    out = torch.empty(st["out"].shape, dtype=torch.float64, device=st["out"].device)
    for at in range(0, st["channels"], 16384):
        w = st["w"][at:at + 16384].double() * st["w_scale"][at:at + 16384].double()[:, None]
        out[:, at:at + 16384] = (st["a"].double() * st["a_scale"].double()[:, None]) @ w.t()
    return out


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    M = case["tokens"]
    if case["op"] == "norm":
        H = case["hidden"]
        width = {"bf16": 2, "f32": 4}
        moved = M * H * (width[case["x"]] + 2 * width[case["residual"]] + 2) + 2 * H
        if case["q"] != "none":
            moved += M * H + 4 * M
        return {"bytes": moved, "flops": 7 * M * H}
    if case["op"] == "route":
        E, K = case["experts"], case["topk"]
        return {"bytes": 4 * M * E + (4 * E if case["bias"] else 0) + 8 * M * K, "flops": 4 * M * E}
    N, K = case["channels"], case["depth"]
    return {"bytes": M * K + N * K + 4 * (M + N) + M * N * {"bf16": 2, "f32": 4}[case["out"]], "flops": 2 * M * N * K}
