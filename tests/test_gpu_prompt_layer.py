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
