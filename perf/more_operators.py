"""The prompt operators of a decoder layer: inputs, plain forms and reference results.

Three operators of this package are described here, each as a small set of cases:

  turn     norms of queries and keys for each head, and the position rotation
  prompt   causal attention over whole prompts, packed one behind the other
  adapt    low-rank adapters of many requests beside a shared projection

``run`` computes a case either with the package's kernels (``own`` true) or in its
plain form: elementary torch operations in fp32 (the rotation's angles in fp64), rounded
once at the end.  ``exact`` gives the operators' definitions in fp64.

turn: token n of position p(n), head h, x its D values:
    y = x / sqrt(mean(x^2) + eps) * weight
and of the first R columns the pairs (i, i + R / 2), or (2 i, 2 i + 1) where they are
interleaved, are turned by the angle p(n) * inv_freq[i].

prompt: sequence b has the tokens offsets[b] .. offsets[b + 1] - 1; each token's queries see
the keys of its sequence up to its own: out = softmax(q K^T / sqrt(D)) V.

adapt: request b has the tokens offsets[b] .. offsets[b + 1] - 1 and the adapter a = ids[b]:
    out = base + scale[a] (x A[a]^T) B[a]^T,
A [adapters, rank, K], B [adapters, N, rank]; a negative id takes base as it is.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 48 streams, each at a position of its own: latency
        dict(name="turn step", op="turn", batch=48, low=1, high=1, first=37, last=16384, q_heads=16,
             heads=16, dim=128, rotary=128, interleaved=False),
        # the prompts of a few streams; half of each head turned, in adjacent pairs
        dict(name="turn prompts", op="turn", batch=7, low=333, high=1999, first=0, last=0, q_heads=32,
             heads=4, dim=64, rotary=32, interleaved=True),
        # a long prefill far into its contexts
        dict(name="turn prefill", op="turn", batch=4, low=16001, high=16384, first=0, last=114687,
             q_heads=32, heads=8, dim=128, rotary=128, interleaved=False),
        # a few short utterances
        dict(name="prompt short", op="prompt", batch=5, low=1, high=77, q_heads=16, heads=8, dim=64),
        # texts of 48 streams, a head of keys for each query head
        dict(name="prompt batch", op="prompt", batch=48, low=37, high=1501, q_heads=16, heads=16, dim=128),
        # prompts of odd lengths, grouped heads
        dict(name="prompt grouped", op="prompt", batch=7, low=333, high=8191, q_heads=32, heads=8, dim=128),
        # long contexts with small heads, a group that does not divide a tile
        dict(name="prompt small heads", op="prompt", batch=3, low=5000, high=16383, q_heads=28, heads=4, dim=64),
        # one long document
        dict(name="prompt document", op="prompt", batch=1, low=32768, high=32768, q_heads=32, heads=8, dim=128),
        # one token for each of 48 requests, each with an adapter of its own
        dict(name="adapt step", op="adapt", batch=48, low=1, high=1, adapters=48, rank=16, K=2048, N=2048),
        # drafted tokens of 64 requests on a few adapters, down projection
        dict(name="adapt drafts", op="adapt", batch=64, low=5, high=5, adapters=8, rank=64, K=8192, N=2048),
        # prompts of a few requests, up projection
        dict(name="adapt prompts", op="adapt", batch=7, low=333, high=1999, adapters=5, rank=32, K=2048, N=8192),
        # a large prefill
        dict(name="adapt prefill", op="adapt", batch=16, low=1777, high=2048, adapters=4, rank=128, K=2048,
             N=8192),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("turn", "prompt", "prompt", "adapt", "adapt"))
    most = [work(c) for c in listed() if c["op"] == op]
    while True:
        c = dict(op=op, batch=log(1, 64))
        if op == "adapt":
            c.update(high=rng.choice((1, log(1, 16), log(1, 4096))), adapters=log(1, 48),
                     rank=rng.choice((8, 16, 24, 32, 64, 128)), K=8 * log(16, 1024), N=8 * log(8, 1024))
        else:
            H = rng.choice((1, 2, 4, 8, 16))
            c.update(heads=H, q_heads=H * rng.choice((1, 2, 3, 4, 7, 8)), dim=rng.choice((64, 128)))
            if op == "turn":
                c.update(high=rng.choice((1, log(1, 16384))), first=0, last=rng.choice((0, log(10, 1 << 20))),
                         rotary=rng.choice((c["dim"], c["dim"], c["dim"] // 2, 48)),
                         interleaved=rng.random() < 0.5)
            else:
                c.update(high=log(1, 32768))
        c["low"] = rng.choice((1, max(1, c["high"] // 2), c["high"]))
        w = work(c)
        if w["bytes"] <= max(m["bytes"] for m in most) and w["flops"] <= max(m["flops"] for m in most):
            return c


def lengths_of(case):
    """Tokens of each sequence: spread over low .. high, the same for every seed."""
    B, lo, hi = case["batch"], case["low"], case["high"]
    if B == 1:
        return [hi]
    return [lo + round((hi - lo) * ((b * 0.6180339887498949 + 0.5) % 1.0)) for b in range(B - 1)] + [hi]


def ids_of(case):
    """Adapter of each request; of more than eight requests every ninth has none."""
    return [-1 if b % 9 == 8 and case["high"] > 1 else b % case["adapters"] for b in range(case["batch"])]


def work(case):
    lens = lengths_of(case)
    n = sum(lens)
    if case["op"] == "turn":
        rows = n * (case["q_heads"] + case["heads"]) * case["dim"]
        return dict(bytes=4 * rows + 4 * n, flops=8 * rows)
    if case["op"] == "prompt":
        seen = sum(m * (m + 1) // 2 for m in lens)
        return dict(bytes=4 * n * (case["q_heads"] + case["heads"]) * case["dim"],
                    flops=4 * case["dim"] * case["q_heads"] * seen)
    ids, r, K, N = ids_of(case), case["rank"], case["K"], case["N"]
    adapted = sum(m for m, a in zip(lens, ids) if a >= 0)
    return dict(bytes=2 * adapted * K + 4 * n * N + 2 * r * (K + N) * len({a for a in ids if a >= 0}),
                flops=2 * adapted * r * (K + N))


# -------------------------------------------------------------------- prepare
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=gen)
    lens = lengths_of(case)
    starts = [0]
    for m in lens:
        starts.append(starts[-1] + m)
    n = starts[-1]
    s = dict(op=case["op"], starts=starts, offsets=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    if case["op"] == "adapt":
        r, K, N, count = case["rank"], case["K"], case["N"], case["adapters"]
        s.update(ids=ids_of(case), id_tensor=torch.tensor(ids_of(case), dtype=torch.int32, device="cuda"),
                 x=torch.randn(n, K, **dev).bfloat16(), base=torch.randn(n, N, **dev).bfloat16(),
                 a=(torch.randn(count, r, K, **dev) * K**-0.5).bfloat16(),
                 b=(torch.randn(count, N, r, **dev) * r**-0.5).bfloat16(),
                 # alpha / rank of different adapters
                 scale=0.25 + 1.75 * torch.rand(count, **dev))
        return s
    Hq, H, D = case["q_heads"], case["heads"], case["dim"]
    # queries, keys and values as the fused projection leaves them: columns of one row per token
    qkv = torch.randn(n, (Hq + 2 * H) * D, **dev)
    if case["op"] == "turn":
        # tokens and channels of different strength
        qkv *= torch.exp(0.5 * torch.randn(n, 1, **dev)) * torch.exp(0.5 * torch.randn(1, qkv.shape[1], **dev))
    else:
        # queries strong enough that a few tokens carry much of the weight
        qkv[:, :Hq * D] *= 2.0
    qkv = qkv.bfloat16().view(n, Hq + 2 * H, D)
    s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:])
    if case["op"] == "turn":
        R = case["rotary"]
        at = torch.randint(case["first"], case["last"] + 1, (len(lens),), **dev).tolist()
        s.update(interleaved=case["interleaved"],
                 positions=torch.cat([torch.arange(p, p + m, device="cuda") for p, m in zip(at, lens)]).int(),
                 inv_freq=10000.0 ** (-torch.arange(0, R, 2, device="cuda").float() / R),
                 q_weight=(1 + 0.2 * torch.randn(D, **dev)).bfloat16(),
                 k_weight=(1 + 0.2 * torch.randn(D, **dev)).bfloat16())
    return s


# ------------------------------------------------------------------------ run
def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    from bit_weight_only_q4_gb300 import q4

    if s["op"] == "turn":
        return q4.q4_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"],
                               eps=EPS, interleaved=s["interleaved"])
    if s["op"] == "prompt":
        return q4.q4_prompt_attention(s["q"], s["k"], s["v"], s["offsets"])
    return q4.q4_lora(s["x"], s["a"], s["b"], s["scale"], s["offsets"], s["id_tensor"], s["base"])


def run_plain(s):
    return dict(turn=plain_turn, prompt=plain_prompt, adapt=plain_adapt)[s["op"]](s)


def plain_turn(s):
    angle = s["positions"].double().view(-1, 1, 1) * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    half = cos.shape[-1]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        if s["interleaved"]:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:2 * half]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out.append(torch.cat((turned, y[..., 2 * half:]), -1).bfloat16())
    return tuple(out)


def plain_prompt(s):
    n, Hq, D = s["q"].shape
    H = s["k"].shape[1]
    G = Hq // H
    out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    for lo, hi in zip(s["starts"], s["starts"][1:]):
        k = s["k"][lo:hi].float().permute(1, 2, 0)               # [H, D, m]
        v = s["v"][lo:hi].float().transpose(0, 1)                # [H, m, D]
        q = s["q"][lo:hi].float().view(hi - lo, H, G, D) / math.sqrt(D)
        step = max(1, (1 << 27) // (Hq * max(1, hi - lo)))       # queries a piece at a time
        for t in range(0, hi - lo, step):
            x = q[t:t + step].transpose(0, 1)                    # [H, T, G, D]
            T = x.shape[1]
            seen = t + T
            scores = (x.reshape(H, T * G, D) @ k[..., :seen]).view(H, T, G, seen)
            later = torch.arange(seen, device="cuda") > torch.arange(t, seen, device="cuda").view(-1, 1)
            scores = scores.masked_fill_(later.view(1, T, 1, seen), -math.inf)
            p = torch.exp_(scores.sub_(scores.amax(-1, keepdim=True)))
            y = (p.view(H, T * G, seen) @ v[:, :seen]).view(H, T, G, D) / p.sum(-1, keepdim=True)
            out[lo + t:lo + seen] = y.transpose(0, 1).reshape(T, Hq, D)
    return out


def plain_adapt(s):
    out = torch.empty_like(s["base"])
    for lo, hi, a in zip(s["starts"], s["starts"][1:], s["ids"]):
        y = s["base"][lo:hi].float()
        if a >= 0:
            y = y + s["scale"][a] * ((s["x"][lo:hi].float() @ s["a"][a].float().T) @ s["b"][a].float().T)
        out[lo:hi] = y
    return out


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    if work(case)["flops"] > 1.2e13:                             # (more than fits some seconds in fp64)
        return None
    s = prepare(case, seed)
    spans = [slice(a, b) for a, b in zip(s["starts"], s["starts"][1:])]
    if case["op"] == "turn":
        got = []
        R, D = case["rotary"], case["dim"]
        first = torch.arange(R // 2, device="cuda")              # the pairs' columns
        one, two = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + R // 2)
        turn = torch.polar(torch.ones(1, 1, dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(), s["inv_freq"].double()))
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for h in range(x.shape[1]):
                z = x[:, h].double()
                z = z * w.double() / ((z.square().sum(-1, keepdim=True) / D + EPS).sqrt())
                pair = torch.complex(z[:, one], z[:, two]) * turn
                z[:, one], z[:, two] = pair.real, pair.imag
                y[:, h] = z
            got.append(y)
        return tuple(got)
    if case["op"] == "adapt":
        out = s["base"].double()
        for span, a in zip(spans, s["ids"]):
            if a >= 0:
                inner = torch.einsum("mk,rk->mr", s["x"][span].double(), s["a"][a].double())
                out[span] += torch.einsum("mr,nr->mn", inner, s["b"][a].double()) * s["scale"][a].double()
        return out
    Hq, H = case["q_heads"], case["heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for span in spans:
        q, k, v = (s[x][span].double() for x in "qkv")
        m = q.shape[0]
        rows = max(64, (1 << 26) // m)
        for h in range(Hq):
            kk, vv = k[:, h * H // Hq], v[:, h * H // Hq]
            for t in range(0, m, rows):
                end = min(m, t + rows)
                a = torch.einsum("td,nd->tn", q[t:end, h], kk[:end]) / math.sqrt(case["dim"])
                a = a + torch.full_like(a, -math.inf).triu(t + 1)
                out[span.start + t:span.start + end, h] = torch.softmax(a, -1) @ vv[:end]
    return out
