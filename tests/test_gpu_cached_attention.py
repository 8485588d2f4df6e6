"""The attention layer on 4-bit weights and a quantised cache, as its command runs it.

The attention of the last step is compared with fp32 attention over K and V read back from
the cache.  Reading back rounds them to bf16, by 2^-9 of a value at most, so scores move by
up to d = 2^-9 max sum |q k| scale and probabilities by e^(2 d) - 1 of themselves; with the
rounding of V, that of the output and of the probabilities (2^-11), per element
    |err| <= 2^-8 |o| + (2^-9 + 2^-9 + 2^-11 + e^(2 d) - 1) sum p |v|
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,kw", [
    (0, dict(streams=5, prompt=77, text=(1, 40), steps=4, hidden=512, q_heads=8, kv_heads=2, head_dim=64)),
    (1, dict(streams=3, prompt=300, text=(17, 130), steps=3, hidden=1024, q_heads=4, kv_heads=4, page=64)),
    (0, dict(streams=1, prompt=1, text=(5, 5), steps=2, hidden=256, q_heads=20, kv_heads=1, page=32)),
])
def test_layer_steps_match_plain_attention(fmt, kw):
    from bit_weight_only_q4_gb300 import cached_attention as C, q4
    q4.device_error_flags(clear=True)
    r = C.run(fmt=fmt, seed=fmt, **kw)
    q, got = C.last_attention(r)
    assert q4.device_error_flags() == 0
    y = q4.q4_linear_int4g128(got.reshape(len(got), -1), *r["layer"].out)
    assert torch.equal(y, r["y"][:, 0])                     # the graph's own result
    # the reference in fp64 on the host
    q, got = q.cpu().double(), got.cpu().double()
    k, v, seen = (t.cpu() for t in C.read_back(r))
    g = q.shape[1] // k.shape[1]
    k, v = (t.double().repeat_interleave(g, 1) for t in (k, v))
    scale = q.shape[2]**-0.5
    s = torch.einsum("bhd,bhnd->bhn", q, k) * scale
    p = s.masked_fill(~seen.unsqueeze(1), -torch.inf).softmax(-1)
    want = torch.einsum("bhn,bhnd->bhd", p, v)
    mag = torch.einsum("bhn,bhnd->bhd", p, v.abs())
    d = 2.0**-9 * float((torch.einsum("bhd,bhnd->bhn", q.abs(), k.abs()) * scale).max())
    bound = 2.0**-8 * want.abs() + (2.0**-8 + 2.0**-11 + math.expm1(2 * d)) * mag
    assert ((got - want).abs() <= bound).all()
    plain, _ = C.plain(r["layer"].project(r["x"])[0][:, 0], *C.read_back(r))
    assert torch.isfinite(plain).all() and plain.shape == want.shape


def test_layer_of_streams_without_a_prefix():
    """The same call without a shared prompt: one sequence of two chunks, then as one chunk."""
    from bit_weight_only_q4_gb300 import cached_attention as C, q4
    gen = torch.Generator("cuda").manual_seed(3)
    H, D, page, n = 2, 64, 16, 50
    x = torch.randn(1, n, 256, device="cuda", generator=gen).bfloat16()
    table = torch.arange(4, dtype=torch.int32, device="cuda").flip(0).contiguous().view(1, 4)
    pos = torch.arange(n, device="cuda")
    slots = (table[0, pos // page] * page + pos % page).int()
    length = lambda m: torch.tensor([m], dtype=torch.int32, device="cuda")
    out = []
    weights = C._weights((4 + 2 * H) * D, 256, gen), C._weights(256, 4 * D, gen)
    for cuts in ((0, n), (0, 21, n)):
        layer = C.CachedAttention(*weights, 4, q4.alloc_kv_cache(0, 4, page, H, D), 0, D)
        y = [layer(x[:, a:b].contiguous(), slots[a:b], table, length(b)) for a, b in zip(cuts, cuts[1:])]
        out.append(torch.cat(y, 1).float().cpu())
    # two roundings of the attention's output to bf16 apart, through one projection of 256 columns
    assert (out[0] - out[1]).abs().max() <= 2.0**-6 * out[0].abs().max()
