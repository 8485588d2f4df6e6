"""Adapters, norms and rotation, prompt attention and the cache together, as a layer runs them: in place on the views
of one projection, prompts packed, then single tokens from a graph.

Each result is compared with the same calls made one by one on tensors of their own (equal, for each is exact in
its inputs), and the attention of the prompts with fp64 and with the attention over the cache, which holds K and V
in 8 bits: there scores move by up to d = scale max sum |q| times half a step of K, values by half a step of V.
"""
import math

import pytest
import torch

from bit_weight_only_q4_gb300 import cached_attention as C
from bit_weight_only_q4_gb300 import q4
from tests.test_gpu_prompt_attention import check, spans_of

pytestmark = pytest.mark.gpu

CASES = [dict(requests=7, prompt=(1, 130), adapters=3, rank=16, steps=5, hidden=512, q_heads=8, kv_heads=2, head_dim=64),
         dict(requests=3, prompt=(200, 300), adapters=2, rank=72, steps=3, hidden=1024, q_heads=4, kv_heads=4, rotary=64),
         dict(requests=1, prompt=(5, 5), adapters=1, rank=8, steps=2, hidden=256, q_heads=20, kv_heads=1, page=32)]


def by_hand(layer, x, offsets, ids, positions):
    """q, k, v of the layer by calls on tensors of their own."""
    n, H, D = layer.q_heads, layer.kv_heads, layer.head_dim
    y = q4.q4_linear_int4g128(x, *layer.qkv)
    y = q4.q4_lora(x, *layer.adapters[0], offsets, ids, y).view(len(x), n + 2 * H, D)
    q, k = q4.q4_norm_rope(y[:, :n].contiguous(), y[:, n:n + H].contiguous(), *layer.turn_by[:2], positions, layer.turn_by[2])
    return q, k, y[:, n + H:].contiguous()


@pytest.mark.parametrize("fmt", [q4.CACHE_INT8, q4.CACHE_INT4])
@pytest.mark.parametrize("kw", CASES, ids=str)
def test_prompts_and_steps(kw, fmt):
    q4.device_error_flags(clear=True)
    r = C.run_requests(fmt=fmt, seed=1, **kw)
    layer, offsets, ids = r["layer"], r["offsets"], r["ids"]
    q, k, v = by_hand(layer, r["prompt_x"], offsets, ids, r["positions"])
    a = q4.q4_prompt_attention(q, k, v, offsets)
    check(a, q, k, v, spans_of(offsets))
    flat = a.view(len(a), -1)
    y = q4.q4_lora(flat, *layer.adapters[1], offsets, ids, q4.q4_linear_int4g128(flat, *layer.out))
    assert torch.equal(r["prompt_y"], y)
    # the last step: its own token is in the cache already, and is written there again
    one = r["step_requests"][0]
    q, k, v = by_hand(layer, r["x"][:, 0].contiguous(), one, ids, r["at"])
    page = 16 * layer.cache.shape[2]
    where = r["table"].gather(1, (r["at"] // page).long().view(-1, 1)).view(-1) * page + r["at"] % page
    before = layer.cache.clone()
    q4.q4_kv_write(k, v, layer.cache, where.int(), fmt)
    assert torch.equal(layer.cache, before)
    a = q4.q4_kv_attention(q.unsqueeze(1), layer.cache, r["table"], r["lengths"], fmt)
    flat = a.view(len(a), -1)
    y = q4.q4_lora(flat, *layer.adapters[1], one, ids, q4.q4_linear_int4g128(flat, *layer.out))
    assert torch.equal(r["y"][:, 0], y)
    assert q4.device_error_flags() == 0


def test_prompts_against_the_attention_over_the_cache():
    kw = dict(CASES[0], prompt=(90, 90), requests=3)
    r = C.run_requests(fmt=q4.CACHE_INT8, seed=2, **kw)
    layer, n = r["layer"], 90
    q, k, v = by_hand(layer, r["prompt_x"], r["offsets"], r["ids"], r["positions"])
    got = q4.q4_prompt_attention(q, k, v, r["offsets"]).double()
    length = torch.full((3,), n, dtype=torch.int32, device="cuda")
    cached = q4.q4_kv_attention(q.view(3, n, layer.q_heads, -1), layer.cache, r["table"], length, q4.CACHE_INT8).double()
    scale = layer.head_dim**-0.5
    step = lambda t: float(t.double().abs().amax()) / 127 * (1 + 2.0**-10)
    d = scale * float(q.double().abs().sum(-1).max()) * step(k) / 2
    top = float(v.double().abs().max())
    # half a step of V, the scores' share, and both sides' roundings
    bound = step(v) / 2 + (math.expm1(2 * d) + 4 * 2.0**-8) * top
    assert (got.view_as(cached) - cached).abs().max() <= bound


def test_a_layer_without_any_of_them_is_what_it_was():
    gen = torch.Generator("cuda").manual_seed(3)
    H, D, n = 2, 64, 50
    weights = C._weights((4 + 2 * H) * D, 256, gen), C._weights(256, 4 * D, gen)
    layer = C.CachedAttention(*weights, 4, q4.alloc_kv_cache(0, 4, 16, H, D), 0, D)
    x = torch.randn(n, 256, device="cuda", generator=gen).bfloat16()
    slots = torch.arange(n, device="cuda").int()
    offsets = torch.tensor([0, 20, n], dtype=torch.int32, device="cuda")
    y = layer.prompt(x, offsets, slots)
    q, k, v = layer.project(x.unsqueeze(0))
    a = q4.q4_prompt_attention(q[0], k, v, offsets)
    assert torch.equal(y, q4.q4_linear_int4g128(a.view(n, -1), *layer.out))


def pieces(tokens, seed, far=None):
    """x, base, q | k | v rows and adapters for `tokens`; far: elements from token to token."""
    gen = torch.Generator("cuda").manual_seed(seed)

    def rows(n):
        t = torch.randn(tokens, n, device="cuda", generator=gen).bfloat16()
        if far is None:
            return t
        wide = torch.empty(tokens * far, device="cuda", dtype=torch.bfloat16).view(tokens, far)[:, :n]
        return wide.copy_(t)

    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)
    return dict(x=rows(256), base=rows(320), qkv=rows(6 * 128).unflatten(1, (6, 128)),
                a=(rand(3, 24, 256) / 16).bfloat16(), b=(rand(3, 320, 24) / 5).bfloat16(), scales=1 + 0.1 * rand(3).abs(),
                w=(1 + 0.1 * rand(128)).bfloat16(), f=10000.0 ** (-torch.arange(64, device="cuda") / 64.0),
                pos=torch.arange(tokens, device="cuda", dtype=torch.int32))


def all_three(p, offsets, ids, in_place=False, stream=None):
    q, k, v = p["qkv"][:, :4], p["qkv"][:, 4:5], p["qkv"][:, 5:]
    to = dict(q_out=q, k_out=k) if in_place else {}
    q, k = q4.q4_norm_rope(q, k, p["w"], p["w"], p["pos"], p["f"], stream=stream, **to)
    return (q, k, q4.q4_prompt_attention(q, k, v, offsets, stream=stream),
            q4.q4_lora(p["x"], p["a"], p["b"], p["scales"], offsets, ids, p["base"], out=p["base"] if in_place else None,
                       stream=stream))


def ints(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# requests of many tokens, of a few, of a few that share adapters
LENS = [([300, 0, 1, 260], [1, -1, 0, 2]), ([7, 9, 8], [0, 1, 2]), ([3] * 12, [0, 1, 2, -1] * 3)]


@pytest.mark.parametrize("lens,ids", LENS, ids=str)
def test_rows_far_apart(lens, ids):
    """Offsets of more than 2^32 bytes (and, at the first lengths, elements) from the tensors' beginnings."""
    n = sum(lens)
    near, far = pieces(n, 5), pieces(n, 5, far=8 * (2**32 // 8 // n + 64) if n > 500 else 8 * (2**31 // 8 // n + 64))
    offsets = ints(*[sum(lens[:i]) for i in range(len(lens) + 1)])
    for in_place in (False, True):
        want, got = all_three(near, offsets, ints(*ids), in_place), all_three(far, offsets, ints(*ids), in_place)
        assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("lens,ids", LENS, ids=str)
def test_streams_at_once_and_chained_launches(lens, ids):
    n = sum(lens)
    offsets, ids = ints(*[sum(lens[:i]) for i in range(len(lens) + 1)]), ints(*ids)
    made = [pieces(n, seed) for seed in range(4)]
    want = [all_three(p, offsets, ids) for p in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        got = [all_three(p, offsets, ids, stream=s) for p, s in zip(made, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for a, b in zip(got, want) for g, w in zip(a, b))
    # launches that begin before the one in front has ended, each reading what that one writes; eager and as a graph
    p = made[0]
    fresh = {k: v.clone() for k, v in p.items()}

    def chain():
        p["base"].copy_(fresh["base"])
        for _ in range(3):
            p["qkv"].copy_(fresh["qkv"])
            out = all_three(p, offsets, ids, in_place=True)
        return out[2], q4.q4_lora(p["x"], p["a"], p["b"], p["scales"], offsets, ids, p["base"])

    plain = [t.clone() for t in chain()]
    q4.set_launch_flags(q4.FLAG_PDL)
    try:
        early = [t.clone() for t in chain()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = chain()
    finally:
        q4.set_launch_flags(0)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(early, plain, out))


def test_threads():
    """Calls of several host threads, each on a stream of its own."""
    from concurrent.futures import ThreadPoolExecutor
    made = [(pieces(sum(lens), 20 + i), ints(*[sum(lens[:j]) for j in range(len(lens) + 1)]), ints(*ids))
            for i, (lens, ids) in enumerate(LENS)]
    want = [all_three(*m) for m in made]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        got = [all_three(*made[i % 3], stream=s) for _ in range(20)][-1]
        s.synchronize()
        return all(torch.equal(g, w) for g, w in zip(got, want[i % 3]))

    with ThreadPoolExecutor(6) as pool:
        assert all(pool.map(work, range(6)))


def test_nothing_but_empty_requests():
    p = pieces(5, 9)
    for offsets, ids in ((ints(0, 0, 0), ints(0, 1)), (ints(5, 5), ints(2)), (ints(*[3] * 41), ints(*[0, 1] * 20))):
        out, to = torch.full((5, 4, 128), 3.0, device="cuda").bfloat16(), torch.full((5, 320), 3.0, device="cuda").bfloat16()
        q4.q4_prompt_attention(p["qkv"][:, :4], p["qkv"][:, 4:5], p["qkv"][:, 5:], offsets, out=out)
        q4.q4_lora(p["x"], p["a"], p["b"], p["scales"], offsets, ids, p["base"], out=to)
        assert (out == 3).all() and (to == 3).all()
    assert q4.device_error_flags() == 0
