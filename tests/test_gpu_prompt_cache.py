"""A layer's prompts and the attention over the cache that they filled, each held to its own error, row by row.

The attention over the cache goes by the values that the cache holds: in fp64 on these (kv_reference.py), per element
    |err| <= 2^-8 |o| + (2^-10 + e^(2 d) - 1) sum p |v|,   d = 2 D 2^-24 scale max sum |q k|
(the result's rounding; probabilities times V's scale as fp16; scores as fp32 sums).  Prompt attention goes by K and V as
they were before: a score differs by scale q (k' - k), which is worked out for every pair, and values by v' - v.
"""
import math

import pytest
import torch

from bit_weight_only_q4_gb300 import cached_attention as C
from bit_weight_only_q4_gb300 import q4
from tests import kv_reference as R
from tests.test_gpu_prompt_attention import want as prompt_want
from tests.test_gpu_prompt_layer import by_hand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [q4.CACHE_INT8, q4.CACHE_INT4])
@pytest.mark.parametrize("kw", [dict(q_heads=8, kv_heads=2, head_dim=64, hidden=512, prompt=(90, 90), requests=3),
                                dict(q_heads=4, kv_heads=4, head_dim=128, hidden=512, prompt=(150, 150), requests=2, page=32)],
                         ids=str)
def test_prompts_and_the_cache_they_filled(kw, fmt):
    r = C.run_requests(fmt=fmt, seed=4, steps=1, adapters=2, rank=16, **kw)
    layer, n, B = r["layer"], kw["prompt"][0], kw["requests"]
    Hq, H, D = layer.q_heads, layer.kv_heads, layer.head_dim
    q, k, v = by_hand(layer, r["prompt_x"], r["offsets"], r["ids"], r["positions"])
    length = torch.full((B,), n, dtype=torch.int32, device="cuda")
    got = q4.q4_prompt_attention(q, k, v, r["offsets"]).double().cpu()
    cached = q4.q4_kv_attention(q.view(B, n, Hq, D), layer.cache, r["table"], length, fmt).double().cpu()
    spans = [(b * n, b * n + n) for b in range(B)]
    ref, tol = (t.cpu() for t in prompt_want(q, k, v, spans, D**-0.5))
    assert ((got - ref).abs() <= tol).all()
    data, table = layer.cache.cpu().numpy(), r["table"].cpu().numpy()
    for b, (lo, hi) in enumerate(spans):
        ck, cv, ok = R.read(data, table[b], n, fmt, D)
        assert ok.all()
        qq = q[lo:hi].double().cpu()
        o, mag = (torch.from_numpy(t) for t in R.attention(qq.numpy(), ck, cv, ok, range(1, n + 1), D**-0.5))
        each = [torch.from_numpy(t).double().repeat_interleave(Hq // H, 1) for t in (ck, cv)]
        kk, vv = (t[lo:hi].double().cpu().repeat_interleave(Hq // H, 1) for t in (k, v))
        d = 2 * D * 2.0**-24 * D**-0.5 * float(torch.einsum("thd,nhd->thn", qq.abs(), each[0].abs()).max())
        exact = 2.0**-8 * o.abs() + (2.0**-10 + math.expm1(2 * d)) * mag
        assert ((cached[b] - o).abs() <= exact).all()
        # what the cache's rounding does to a row: its largest change of a score, and its mean change of v
        seen = torch.ones(n, n, dtype=torch.bool).tril().unsqueeze(1)
        e = (torch.einsum("thd,nhd->thn", qq, each[0] - kk).abs() * D**-0.5).masked_fill(~seen, 0).amax(-1, keepdim=True)
        p = (torch.einsum("thd,nhd->thn", qq, kk) * D**-0.5).masked_fill(~seen, -torch.inf).softmax(-1)
        bound = torch.einsum("thn,nhd->thd", p, (each[1] - vv).abs()) + torch.expm1(2 * e) * torch.einsum("thn,nhd->thd", p, each[1].abs())
        assert ((ref[lo:hi] - o).abs() <= bound + 1e-12).all()
        assert ((got[lo:hi] - cached[b]).abs() <= bound + exact + tol[lo:hi]).all()
        if fmt == q4.CACHE_INT8:                             # (zeros in a row's place would be seen)
            assert (o.abs() > bound + exact).any(-1).all()
