"""Measured cases of the operators beside the projections and the LM head: log
probabilities of given tokens with entropy and top alternatives, and low-rank
adapters of many requests, added to a projection's output or computed with the
int8 projection itself.

``run`` computes each operator in its plain form (elementary torch operations),
or, where ``own`` is true, by the library's calls.

The definitions, which both sides follow:

* log probabilities: of a row of logits l, a NaN counts as -inf and +inf as the largest
  finite fp32 value.  lse = log(sum exp(l)).  A token's log probability is l[token] - lse,
  -inf where l[token] is -inf; its rank is how many stand before it: larger logits, and equal
  ones of a lower index.  Entropy = -sum p log p, 0 for a row with nothing in it.  The top
  alternatives are the K largest logits above -inf, ties to the lowest index, with their log
  probabilities; where there are fewer, id -1 and -inf stand behind them.  A token below 0
  asks for nothing: log probability 0, rank -1.
* adapters: d[m] = B[i] (scale[i] A[i] x[m]) for the adapter i of token m, 0 where i is not
  one of the adapters; out = base + d, rounded once.
* the int8 projection with adapters: base[m,n] = a_scale[m] w_scale[n] sum_k a[m,k] w[n,k].
"""
import math

import torch

own = False

DEVICE = "cuda"
F32_MAX = torch.finfo(torch.float32).max
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


# ---- the cases --------------------------------------------------------------
def _logprobs(tokens, vocab, logits, topk, pad=0, masked=0.0, name=None):
    return _named(name, op="logprobs", tokens=tokens, vocab=vocab, logits=logits, topk=topk, pad=pad, masked=masked)


def _lora(tokens, requests, bare, adapters, rank, depth, channels, out, int8=False, name=None):
    return _named(name, op="int8_lora" if int8 else "lora", tokens=tokens, requests=requests, bare=bare, adapters=adapters,
                  rank=rank, depth=depth, channels=channels, out=out)


def _named(name, **case):
    return case if name is None else dict(case, name=name)


def listed():
    return [
        # one decoded token over the whole vocabulary, with the alternatives that an API answers with
        _logprobs(1, 157184, "f32", 20, name="logprobs_decode_1"),
        # the four positions of a verify window: the drafted tokens' probabilities and the best token of each
        _logprobs(4, 157184, "f32", 1, name="logprobs_verify_4"),
        # a batch of constrained requests: bf16 logits, most of the vocabulary masked
        _logprobs(64, 157184, "bf16", 5, masked=0.7, name="logprobs_batch_64"),
        # a prompt over an odd vocabulary whose rows are padded, no alternatives
        _logprobs(301, 32771, "bf16", 0, pad=61, name="logprobs_ragged_301"),
        # every position of a long prompt
        _logprobs(2048, 157184, "f32", 5, name="logprobs_prompt_2048"),
        # one decoded token's adapter beside a dense projection
        _lora(1, 1, 0, 8, 16, 2560, 2560, "bf16", name="lora_decode_1"),
        # a decode batch of 64 requests, nearly each with an adapter of its own
        _lora(64, 64, 6, 64, 16, 2560, 2560, "bf16", name="lora_batch_64"),
        # four requests' adapters of the LM head on fp32 logits
        _lora(4, 4, 0, 8, 16, 2560, 157184, "f32", name="lora_head_4"),
        # prefill chunks of five requests, wide adapters
        _lora(2048, 5, 1, 8, 64, 2560, 2560, "bf16", name="lora_chunk_2048"),
        # the verify windows of eight requests through an int8 projection with adapters
        _lora(32, 8, 1, 16, 16, 2560, 2560, "bf16", int8=True, name="int8_lora_verify_32"),
        # no size a multiple of anything
        _lora(77, 9, 2, 5, 13, 769, 2563, "f32", int8=True, name="int8_lora_ragged_77"),
        # a long chunk of six requests through an int8 projection with adapters
        _lora(2048, 6, 1, 8, 16, 2560, 2560, "bf16", int8=True, name="int8_lora_chunk_2048"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _rough(rng, lo, hi):
    """As _log; half of them are made multiples of 64 where they are large enough."""
    n = _log(rng, lo, hi)
    return n // 64 * 64 if n >= 128 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["logprobs", "lora", "int8_lora"])
    if op == "logprobs":
        vocab = _rough(rng, 2, 262144)
        tokens = min(_log(rng, 1, 4096), 2048 * 157184 // vocab)
        return _logprobs(tokens, vocab, rng.choice(["bf16", "f32"]), rng.choice([0, 1, 5, rng.randint(2, 32)]),
                         rng.choice([0, 0, rng.randint(1, 128)]), rng.choice([0.0, 0.0, 0.7, 0.99]))
    rank = rng.choice([8, 16, 32, 64, rng.randint(1, 128)])
    depth = _rough(rng, 16, 8192)
    tokens = _log(rng, 1, 2048)
    channels = _rough(rng, 16, max(16, min(16384, 2048 * 2560 * 2560 // (tokens * depth))))
    requests = _log(rng, 1, min(tokens, 64))
    return _lora(tokens, requests, rng.randint(0, requests // 3), _log(rng, 1, 64), rank, depth, channels,
                 rng.choice(["bf16", "f32"]), int8=op == "int8_lora")


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
    if case["op"] == "logprobs":
        V, K = case["vocab"], case["topk"]
        # what a head gives: most logits in a broad bell, one token well above it in confident rows and lost in
        # it in others; sampled tokens are mostly that one
        full = 2.0 * normal(M, V + case["pad"])
        peak = torch.randint(V, (M, 1), generator=g, device=DEVICE)
        full.scatter_add_(1, peak, 24.0 * uniform(M, 1))
        if case["masked"] > 0.0:  # tokens that a grammar excludes; now and then none is left
            for at in range(0, M, 256):
                part = full[at:at + 256]
                gone = uniform(*part.shape) < case["masked"]
                gone |= uniform(part.shape[0], 1) < 0.02
                part.masked_fill_(gone, -INF)
        st["logits"] = full.to(TYPES[case["logits"]])[:, :V]
        other = torch.randint(V, (M, 1), generator=g, device=DEVICE)
        tokens = torch.where(uniform(M, 1) < 0.7, peak, other)
        tokens = torch.where(uniform(M, 1) < 0.05, -1, tokens) if M > 1 else tokens  # positions with nothing to ask for
        st["tokens_given"] = tokens[:, 0].to(torch.int32)
        st["logprob"], st["rank_out"], st["entropy"] = (empty((M,), t) for t in (torch.float32, torch.int32, torch.float32))
        st["topk_ids"] = empty((M, K), torch.int32) if K else None
        st["topk_logprob"] = empty((M, K), torch.float32) if K else None
        return st
    L, r, K, N = case["adapters"], case["rank"], case["depth"], case["channels"]
    x = normal(M, K) * torch.exp(0.3 * normal(M, 1))
    st["x"] = x.to(torch.bfloat16)
    st["a"] = (normal(L, r, K) / math.sqrt(K)).to(torch.bfloat16)
    st["b"] = (0.3 * normal(L, N, r) / math.sqrt(r)).to(torch.bfloat16)
    st["scale"] = 0.5 + 1.5 * uniform(L)
    # a request's tokens follow one another; requests differ in length, and take the adapters in turn
    cuts = torch.randperm(M - 1, generator=g, device=DEVICE)[: case["requests"] - 1] if M > 1 else empty((0,), torch.int64)
    starts = torch.zeros(M, dtype=torch.int64, device=DEVICE)
    starts[cuts + 1] = 1
    owner = torch.randperm(L, generator=g, device=DEVICE)[torch.arange(case["requests"] - case["bare"], device=DEVICE) % L]
    owner = torch.cat([owner, torch.full((case["bare"],), -1, dtype=torch.int64, device=DEVICE)])
    owner = owner[torch.randperm(case["requests"], generator=g, device=DEVICE)]
    st["ids"] = owner[torch.cumsum(starts, 0)].to(torch.int32)
    st["out_rows"] = empty((M, N), TYPES[case["out"]])
    if case["op"] == "lora":
        st["base"] = normal(M, N).to(TYPES[case["out"]])
    else:
        st["codes"], st["codes_scale"] = _rows_to_int8(x)
        st["w"], st["w_scale"] = _rows_to_int8(normal(N, K) / math.sqrt(K))
    return st


# ---- one pass -------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    return {"logprobs": _plain_logprobs, "lora": _plain_lora, "int8_lora": _plain_int8_lora}[st["op"]](st)


def _run_own(st):
    from mxfp4_weight_streaming_amd import binding as moe
    if st["op"] == "logprobs":
        if "workspace" not in st:  # a program keeps one
            st["workspace"] = moe.logprobs_workspace(st["tokens"], st["vocab"], st["topk"])
        moe.moe_token_logprobs(st["logits"], st["tokens_given"], st["logprob"], st["rank_out"], st["entropy"],
                               st["topk_ids"], st["topk_logprob"], st["workspace"])
        return st["logprob"], st["rank_out"], st["entropy"], st["topk_ids"], st["topk_logprob"]
    if "adapters_held" not in st:  # a program describes its adapters once, and keeps a workspace
        st["adapters_held"] = moe.lora(st["a"], st["b"], st["scale"])
        st["workspace"] = moe.lora_workspace(st["adapters_held"], st["tokens"])
    if st["op"] == "lora":
        moe.moe_lora_add(st["adapters_held"], st["x"], st["ids"], st["base"], st["out_rows"], st["workspace"])
    else:
        moe.moe_int8_linear_lora(st["codes"], st["codes_scale"], st["w"], st["w_scale"], st["adapters_held"], st["x"],
                                 st["ids"], st["out_rows"], st["workspace"])
    return st["out_rows"]


def _plain_logprobs(st):
    M, V = st["logits"].shape
    K, tokens = st["topk"], st["tokens_given"].long()
    x = st["logits"].float() + 0.0  # no -0, which is equal to 0
    x = torch.where(torch.isnan(x), -INF, x).clamp(max=F32_MAX)
    best, where = x.max(1, keepdim=True)
    empty = best[:, 0] == -INF
    # in 64 bits and without the largest: a confident row's log probability is what the others are beside its 1
    d = x.double() - torch.where(best == -INF, 0.0, best).double()
    e = torch.exp(d)
    others = e.scatter(1, where, 0.0).sum(1)
    log_total = torch.where(empty, 0.0, torch.log1p(others))
    mean = torch.where(e == 0, 0.0, d * e).sum(1) / (1.0 + others)
    entropy = torch.where(empty, 0.0, log_total - mean).float()

    def log_p(values, at):  # of d's values
        return torch.where(values == -INF, -INF, values - log_total.view(at)).float()

    asked = tokens.clamp(min=0)[:, None]
    logprob = torch.where(tokens < 0, 0.0, log_p(d.gather(1, asked)[:, 0], (M,)))
    mine = x.gather(1, asked)
    index = torch.arange(V, device=x.device)
    rank = ((x > mine) | ((x == mine) & (index < asked))).sum(1)
    rank = torch.where(tokens < 0, -1, rank).to(torch.int32)
    if K == 0:
        return logprob, rank, entropy, None, None
    # keys that are all different: the value's order, then the index backwards
    bits = x.view(torch.int32)
    keys = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + ((1 << 32) - 1 - index)
    n = min(K, V)
    ids = (1 << 32) - 1 - (torch.topk(keys, n, dim=1).values & 0xFFFFFFFF)
    values = d.gather(1, ids)
    ids = torch.where(values == -INF, -1, ids).to(torch.int32)
    values = log_p(values, (M, 1))
    return (logprob, rank, entropy, torch.nn.functional.pad(ids, (0, K - n), value=-1),
            torch.nn.functional.pad(values, (0, K - n), value=-INF))


def _plain_delta(st):
    L, r, K = st["a"].shape
    N = st["b"].shape[1]
    M = st["x"].shape[0]
    mine = st["ids"][:, None] == torch.arange(L, device=st["ids"].device)
    u = (st["x"].float() @ st["a"].float().view(L * r, K).t()).view(M, L, r)
    u = torch.where(mine[:, :, None], u * st["scale"][:, None], 0.0)
    return u.view(M, L * r) @ st["b"].float().transpose(1, 2).reshape(L * r, N)


def _plain_lora(st):
    return (st["base"].float() + _plain_delta(st)).to(st["out_rows"].dtype)


def _plain_int8_lora(st):
    acc = st["codes"].float() @ st["w"].float().t()
    return (acc * st["codes_scale"][:, None] * st["w_scale"] + _plain_delta(st)).to(st["out_rows"].dtype)


# ---- the definitions in 64 bits ----------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_logprobs(st) if case["op"] == "logprobs" else _exact_lora(st)


def _exact_logprobs(st):
    M, V = st["logits"].shape
    K = st["topk"]
    logprob, entropy, top = [], [], []
    for at in range(0, M, 128):
        x = torch.nan_to_num(st["logits"][at:at + 128].double(), nan=-INF, posinf=F32_MAX, neginf=-INF)
        # log(1 + what the others are beside the largest): a difference of logarithms would lose a confident row's
        most, first = x.max(1, keepdim=True)
        rest = torch.logsumexp(x.scatter(1, first, -INF), 1, keepdim=True)
        logp = torch.where(torch.isinf(x), -INF, (x - most) - torch.log1p(torch.exp(rest - most)))
        t = st["tokens_given"][at:at + 128].long()
        row = torch.arange(len(t), device=t.device)
        logprob.append(torch.where(t >= 0, logp[row, t % V], torch.zeros_like(logp[:, 0])))
        entropy.append(torch.special.entr(torch.exp(logp)).sum(1))
        best = torch.sort(torch.topk(logp, min(K, V), 1, sorted=False).values, 1, descending=True).values
        top.append(torch.cat([best, torch.full((len(t), K - best.shape[1]), -INF, dtype=torch.float64, device=t.device)], 1))
    return torch.cat(logprob), None, torch.cat(entropy), None, torch.cat(top) if K else None


def _exact_lora(st):
    if st["op"] == "lora":
        out = st["base"].double()
    else:
        out = (st["codes"].double() * st["codes_scale"].double()[:, None]) @ (st["w"].double() * st["w_scale"].double()[:, None]).t()
    for i in torch.unique(st["ids"]).tolist():
        if i < 0:
            continue
        rows = torch.nonzero(st["ids"] == i)[:, 0]
        low = torch.matmul(st["x"][rows].double(), st["a"][i].double().t())
        out[rows] += float(st["scale"][i]) * torch.matmul(low, st["b"][i].double().t())
    return out


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    M = case["tokens"]
    if case["op"] == "logprobs":
        V, K = case["vocab"], case["topk"]
        return {"bytes": M * V * {"bf16": 2, "f32": 4}[case["logits"]] + M * (16 + 8 * K), "flops": 6 * M * V}
    N, K, r = case["channels"], case["depth"], case["rank"]
    used = min(case["requests"] - case["bare"], case["adapters"])
    width = {"bf16": 2, "f32": 4}[case["out"]]
    moved = 2 * M * K + used * (2 * r * (K + N) + 4) + 4 * M + M * N * width
    flops = 2 * M * r * (K + N)
    if case["op"] == "lora":
        return {"bytes": moved + M * N * width, "flops": flops}
    return {"bytes": moved + M * K + N * K + 4 * (M + N), "flops": flops + 2 * M * N * K}
