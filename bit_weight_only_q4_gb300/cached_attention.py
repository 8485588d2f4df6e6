"""An attention layer of a decoder on 4-bit weights and a quantised key/value cache, and a
command that runs one: streams that share a prompt, a text of their own for each, then
single tokens from a captured CUDA graph.

    python -m bit_weight_only_q4_gb300.cached_attention [--streams 48] [--prompt 1501] ...
    python -m bit_weight_only_q4_gb300.cached_attention --requests 24 [--adapters 4] ...

The layer is two projections around three calls: the rows of K and V are written into the
cache straight from the fused q|k|v projection's output, attention reads them where they
lie (what the streams share once for all of them), and the output projection follows.
Beside the projections there may be low-rank adapters, another for each request; between the
projection and the cache, norms of q and k and the position rotation, in place.  Whole prompts
of several requests, packed one behind the other, go through prompt(): their attention reads
K and V as the projection left them, not by way of the cache.  Positions are the caller's: a
model that turns q and k in a way of its own calls project(), turns them, and hands them to attend().
"""
from __future__ import annotations

import argparse

import torch

from . import q4


class CachedAttention:
    """Weights are (qweight, scale, min) of q4_linear_int4g128, qkv with its rows in the order
    q heads, k heads, v heads; the cache is one of q4.alloc_kv_cache.

    turn: norms and rotation of q and k, as q4_norm_rope takes them: (q_weight, k_weight, inv_freq),
    weights None for no norm.  adapters: (of qkv, of out), each (a, b, scales) as q4_lora takes them, or
    None; calls then name their requests as (offsets, ids), and one that names none has the projections alone.  An
    adapter of qkv is one for all of its rows: those of q, k and v apart are stacked, A's rows one below the
    other and B's columns side by side with zeros in the others' rows, up to a rank of 128 together."""

    def __init__(self, qkv, out, q_heads: int, cache: torch.Tensor, fmt: int, head_dim: int, turn=None, adapters=None,
                 eps=1e-6, interleaved=False):
        self.qkv, self.out = qkv, out
        self.q_heads, self.kv_heads, self.head_dim = q_heads, cache.shape[1], head_dim
        self.cache, self.fmt = cache, fmt
        self.turn_by, self.adapters, self.eps, self.interleaved = turn, adapters or (None, None), eps, interleaved

    def _linear(self, x, weights, adapters, requests):
        """x [tokens, columns] through a projection and, beside it, the requests' adapters."""
        y = q4.q4_linear_int4g128(x, *weights)
        if adapters is not None and requests is not None:
            q4.q4_lora(x, *adapters, *requests, y, out=y)
        return y

    def project(self, x, requests=None):
        """x bf16 [batch, tokens, hidden] -> q [batch, tokens, q_heads, D], and k and v
        [batch * tokens, kv_heads, D]: three views of one projection."""
        B, T, _ = x.shape
        n, H, D = self.q_heads, self.kv_heads, self.head_dim
        y = self._linear(x.view(B * T, -1), self.qkv, self.adapters[0], requests).view(B * T, n + 2 * H, D)
        return y[:, :n].view(B, T, n, D), y[:, n:n + H], y[:, n + H:]

    def turn(self, q, k, positions):
        """Norms and rotation of q and k where they lie (positions int32 [batch * tokens])."""
        if self.turn_by is not None:
            q4.q4_norm_rope(q, k, *self.turn_by[:2], positions, self.turn_by[2], eps=self.eps,
                            interleaved=self.interleaved, q_out=q, k_out=k)

    def __call__(self, x, slots, table, lengths, prefix_pages=None, prefix_len=0, positions=None, requests=None):
        """project(), turn() and attend()."""
        q, k, v = self.project(x, requests)
        self.turn(q, k, positions)
        return self.attend(q, k, v, slots, table, lengths, prefix_pages, prefix_len, requests)

    def attend(self, q, k, v, slots, table, lengths, prefix_pages=None, prefix_len=0, requests=None):
        """The new tokens' rows go to `slots` (int32 [batch * tokens]; negative: not cached again);
        `lengths` counts them.  With a prefix, table and lengths describe what lies behind it."""
        B, T = q.shape[:2]
        q4.q4_kv_write(k, v, self.cache, slots, self.fmt)
        if prefix_pages is None:
            a = q4.q4_kv_attention(q, self.cache, table, lengths, self.fmt)
        else:
            a = q4.q4_kv_attention_shared(q, self.cache, prefix_pages, prefix_len, table, lengths, self.fmt)
        return self._linear(a.view(B * T, -1), self.out, self.adapters[1], requests).view(B, T, -1)

    def prompt(self, x, offsets, slots, positions=None, ids=None):
        """Whole prompts: x [tokens, hidden], those of prompt b in the rows offsets[b] .. offsets[b + 1] - 1 (every
        row belongs to one); K and V go to the cache's `slots` for the tokens to come.  ids: the adapter of
        each prompt."""
        requests = None if ids is None else (offsets, ids)
        q, k, v = self.project(x.unsqueeze(0), requests)
        self.turn(q, k, positions)
        q4.q4_kv_write(k, v, self.cache, slots, self.fmt)
        a = q4.q4_prompt_attention(q[0], k, v, offsets)
        return self._linear(a.view(len(a), -1), self.out, self.adapters[1], requests)


def _weights(rows: int, cols: int, gen):
    w = torch.randn(rows, cols, device="cuda", generator=gen, dtype=torch.float32) * cols**-0.5
    return q4.q4_quantize_int4g128(w.bfloat16())


def run(streams=48, prompt=1501, text=(40, 200), steps=16, hidden=2048, q_heads=16, kv_heads=16, head_dim=128,
        page=16, fmt=q4.CACHE_INT8, seed=0):
    """Prompt, texts and `steps` single tokens of random activations.  Returns a dict with the
    layer, the last step's input and output, page tables and lengths, and the time of a step in us."""
    gen = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen).bfloat16()
    ints = lambda a: torch.as_tensor(a, dtype=torch.int32, device="cuda")
    texts = [text[0] + (text[1] - text[0]) * b // max(1, streams - 1) for b in range(streams)]
    pages_of = lambda n: -(-n // page)
    width = pages_of(max(texts) + steps)
    shared = ints(range(pages_of(prompt)))
    table = (ints(range(streams * width)) + shared.numel()).view(streams, width)
    cache = q4.alloc_kv_cache(fmt, shared.numel() + streams * width, page, kv_heads, head_dim)
    layer = CachedAttention(_weights((q_heads + 2 * kv_heads) * head_dim, hidden, gen),
                            _weights(hidden, q_heads * head_dim, gen), q_heads, cache, fmt, head_dim)

    # the shared prompt, as one sequence
    pos = torch.arange(prompt, device="cuda")
    layer(rand(1, prompt, hidden), (shared[pos // page] * page + pos % page).int(), shared.view(1, -1), ints([prompt]))
    # each stream's text behind it; rows that fill the batch up to the longest stand before the
    # text: they are not cached, and their results go unused
    most = max(texts)
    at = torch.arange(most, device="cuda") - most + ints(texts).view(-1, 1)
    slots = torch.where(at >= 0, table.gather(1, at.clamp(min=0) // page) * page + at % page, -1).int()
    lengths = ints(texts)
    layer(rand(streams, most, hidden), slots.view(-1), table, lengths, shared, prompt)

    # single tokens: the step's tensors are updated in place, so one graph serves every step
    x = rand(streams, 1, hidden)
    slots = torch.empty(streams, dtype=torch.int32, device="cuda")

    def advance():
        where = table.gather(1, (lengths // page).long().view(-1, 1)).view(-1)
        torch.add(where * page, lengths % page, out=slots)
        lengths.add_(1)

    advance()
    y = layer(x, slots, table, lengths, shared, prompt)    # (makes the workspaces)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer(x, slots, table, lengths, shared, prompt)    # the same token once more
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = layer(x, slots, table, lengths, shared, prompt)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(steps - 1):
            x.copy_(rand(streams, 1, hidden))
            advance()
            begin.record()
            graph.replay()
            end.record()
            end.synchronize()
            times.append(begin.elapsed_time(end) * 1e3)
    torch.cuda.current_stream().wait_stream(stream)
    return dict(layer=layer, x=x, y=y, shared=shared, prompt=prompt, table=table, lengths=lengths,
                us_per_step=sorted(times)[len(times) // 2] if times else float("nan"))


def run_requests(requests=24, prompt=(37, 400), adapters=4, rank=16, steps=16, hidden=2048, q_heads=16, kv_heads=16,
                 head_dim=128, rotary=None, page=16, fmt=q4.CACHE_INT8, seed=0):
    """The prompts of several requests in one call, then `steps` single tokens of each, with norms, rotation and an
    adapter for each request.  Returns a dict with the layer, the prompts' input and output, the last step's,
    page table and lengths, and the time of the prompts and of a step in us."""
    gen = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)
    ints = lambda a: torch.as_tensor(a, dtype=torch.int32, device="cuda")
    lens = [prompt[0] + (prompt[1] - prompt[0]) * b // max(1, requests - 1) for b in range(requests)]
    width = -(-(max(lens) + steps) // page)
    table = ints(range(requests * width)).view(requests, width)
    cache = q4.alloc_kv_cache(fmt, requests * width, page, kv_heads, head_dim)
    rows, cols, R = (q_heads + 2 * kv_heads) * head_dim, q_heads * head_dim, rotary or head_dim
    adapter = lambda K, N: ((rand(adapters, rank, K) * K**-0.5).bfloat16(), (rand(adapters, N, rank) * rank**-0.5).bfloat16(),
                            torch.full((adapters,), 0.5, device="cuda"))
    turn = ((1 + 0.1 * rand(head_dim)).bfloat16(), (1 + 0.1 * rand(head_dim)).bfloat16(),
            10000.0 ** (-torch.arange(0, R, 2, device="cuda").float() / R))
    layer = CachedAttention(_weights(rows, hidden, gen), _weights(hidden, cols, gen), q_heads, cache, fmt, head_dim, turn,
                            (adapter(hidden, rows), adapter(cols, hidden)))
    ids = ints([b % (adapters + 1) - 1 for b in range(requests)])        # (one in so many has none)

    lengths, begins = ints(lens), torch.cumsum(ints([0] + lens), 0).int()
    positions = torch.cat([torch.arange(n, device="cuda") for n in lens]).int()
    of = torch.repeat_interleave(torch.arange(requests, device="cuda"), lengths.long())
    slots = (table[of, positions.long() // page] * page + positions % page).int()
    x = rand(len(positions), hidden).bfloat16()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):                                      # (the second is timed; it writes the same rows again)
        begin.record()
        y = layer.prompt(x, begins, slots, positions, ids)
        end.record()
    end.synchronize()
    r = dict(layer=layer, prompt_x=x, prompt_y=y, offsets=begins, slots=slots, positions=positions, ids=ids, table=table,
             lengths=lengths, us_prompts=begin.elapsed_time(end) * 1e3)

    # single tokens: the step's tensors are updated in place, so one graph serves every step
    x, one = rand(requests, 1, hidden).bfloat16(), torch.arange(requests + 1, device="cuda").int()
    slots, at = torch.empty(requests, dtype=torch.int32, device="cuda"), torch.empty(requests, dtype=torch.int32, device="cuda")
    step = lambda: layer(x, slots, table, lengths, positions=at, requests=(one, ids))

    def advance():
        at.copy_(lengths)
        torch.add(table.gather(1, (lengths // page).long().view(-1, 1)).view(-1) * page, lengths % page, out=slots)
        lengths.add_(1)

    advance()
    y = step()                                              # (makes the workspaces)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    times = []
    with torch.cuda.stream(stream):
        step()                                              # the same token once more
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = step()
        for _ in range(steps - 1):
            x.copy_(rand(requests, 1, hidden))
            advance()
            begin.record()
            graph.replay()
            end.record()
            end.synchronize()
            times.append(begin.elapsed_time(end) * 1e3)
    torch.cuda.current_stream().wait_stream(stream)
    return dict(r, x=x, y=y, at=at, step_requests=(one, ids),
                us_per_step=sorted(times)[len(times) // 2] if times else float("nan"))


def read_back(r):
    """K and V of every stream's tokens, prompt first, as bf16 values [streams, kv_heads, n, D], and
    which of them each stream has [streams, n]."""
    layer, D = r["layer"], r["layer"].head_dim
    one = torch.full((1,), r["prompt"], dtype=torch.int32, device="cuda")
    pre = q4.q4_kv_read(layer.cache, r["shared"].view(1, -1), one, r["prompt"], D, layer.fmt)
    most = int(r["lengths"].max())
    own = q4.q4_kv_read(layer.cache, r["table"], r["lengths"], most, D, layer.fmt)
    k, v = (torch.cat((p.expand(len(o), -1, -1, -1), o), 1).transpose(1, 2) for p, o in zip(pre, own))
    return k, v, torch.arange(k.shape[2], device="cuda") < r["prompt"] + r["lengths"].view(-1, 1)


def plain(q, k, v, seen):
    """Attention of q [streams, q_heads, D] in fp32: (out, probabilities [streams, q_heads, n])."""
    k, v = (t.float().repeat_interleave(q.shape[1] // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("bhd,bhnd->bhn", q.float(), k) * q.shape[2]**-0.5
    p = s.masked_fill(~seen.unsqueeze(1), -torch.inf).softmax(-1)
    return torch.einsum("bhn,bhnd->bhd", p, v), p


def last_attention(r):
    """q and the attention's output [streams, q_heads, D] of a run's last step, once more."""
    layer = r["layer"]
    q, _, _ = layer.project(r["x"])
    a = q4.q4_kv_attention_shared(q, layer.cache, r["shared"], r["prompt"], r["table"], r["lengths"], layer.fmt)
    return q[:, 0], a[:, 0]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--streams", type=int, default=48)
    ap.add_argument("--prompt", type=int, default=1501)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--int4-cache", action="store_true")
    ap.add_argument("--requests", type=int, default=0, help="prompts of so many requests, each with an adapter, instead")
    ap.add_argument("--adapters", type=int, default=4)
    args = ap.parse_args()
    if args.requests > 0:
        r = run_requests(args.requests, adapters=args.adapters, steps=args.steps,
                         fmt=q4.CACHE_INT4 if args.int4_cache else q4.CACHE_INT8)
        print(f"{args.requests} requests, {len(r['positions'])} tokens of prompts in {r['us_prompts']:.1f} us, then "
              f"{r['us_per_step']:.1f} us a step of one layer")
        return
    r = run(args.streams, args.prompt, steps=args.steps, fmt=q4.CACHE_INT4 if args.int4_cache else q4.CACHE_INT8)
    q, got = last_attention(r)
    want, _ = plain(q, *read_back(r))
    print(f"{args.streams} streams, prompt of {args.prompt}, {int(r['lengths'].max())} tokens at most behind it: "
          f"{r['us_per_step']:.1f} us a step of one layer; largest difference from plain attention "
          f"{float((got.float() - want).abs().max()):.2e} (values up to {float(want.abs().max()):.2e})")


if __name__ == "__main__":
    main()
