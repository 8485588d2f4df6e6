"""An attention layer of a decoder on 4-bit weights and a quantised key/value cache, and a
command that runs one: streams that share a prompt, a text of their own for each, then
single tokens from a captured CUDA graph.

    python -m bit_weight_only_q4_gb300.cached_attention [--streams 48] [--prompt 1501] ...

The layer is two projections around three calls: the rows of K and V are written into the
cache straight from the fused q|k|v projection's output, attention reads them where they
lie (what the streams share once for all of them), and the output projection follows.
Positions are the caller's: a model with rotary positions calls project(), turns q and k, and
hands them to attend().
"""
from __future__ import annotations

import argparse

import torch

from . import q4


class CachedAttention:
    """Weights are (qweight, scale, min) of q4_linear_int4g128, qkv with its rows in the order
    q heads, k heads, v heads; the cache is one of q4.alloc_kv_cache."""

    def __init__(self, qkv, out, q_heads: int, cache: torch.Tensor, fmt: int, head_dim: int):
        self.qkv, self.out = qkv, out
        self.q_heads, self.kv_heads, self.head_dim = q_heads, cache.shape[1], head_dim
        self.cache, self.fmt = cache, fmt

    def project(self, x):
        """x bf16 [batch, tokens, hidden] -> q [batch, tokens, q_heads, D], and k and v
        [batch * tokens, kv_heads, D]: three views of one projection."""
        B, T, _ = x.shape
        n, H, D = self.q_heads, self.kv_heads, self.head_dim
        y = q4.q4_linear_int4g128(x.view(B * T, -1), *self.qkv).view(B * T, n + 2 * H, D)
        return y[:, :n].view(B, T, n, D), y[:, n:n + H], y[:, n + H:]

    def __call__(self, x, slots, table, lengths, prefix_pages=None, prefix_len=0):
        """project() and attend()."""
        return self.attend(*self.project(x), slots, table, lengths, prefix_pages, prefix_len)

    def attend(self, q, k, v, slots, table, lengths, prefix_pages=None, prefix_len=0):
        """The new tokens' rows go to `slots` (int32 [batch * tokens]; negative: not cached again);
        `lengths` counts them.  With a prefix, table and lengths describe what lies behind it."""
        B, T = q.shape[:2]
        q4.q4_kv_write(k, v, self.cache, slots, self.fmt)
        if prefix_pages is None:
            a = q4.q4_kv_attention(q, self.cache, table, lengths, self.fmt)
        else:
            a = q4.q4_kv_attention_shared(q, self.cache, prefix_pages, prefix_len, table, lengths, self.fmt)
        return q4.q4_linear_int4g128(a.view(B * T, -1), *self.out).view(B, T, -1)


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
    args = ap.parse_args()
    r = run(args.streams, args.prompt, steps=args.steps, fmt=q4.CACHE_INT4 if args.int4_cache else q4.CACHE_INT8)
    q, got = last_attention(r)
    want, _ = plain(q, *read_back(r))
    print(f"{args.streams} streams, prompt of {args.prompt}, {int(r['lengths'].max())} tokens at most behind it: "
          f"{r['us_per_step']:.1f} us a step of one layer; largest difference from plain attention "
          f"{float((got.float() - want).abs().max()):.2e} (values up to {float(want.abs().max()):.2e})")


if __name__ == "__main__":
    main()
