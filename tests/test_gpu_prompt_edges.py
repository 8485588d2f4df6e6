"""Causal attention over packed prompts (q4_prompt_attention): scores, values and units at the ends of their ranges."""
from __future__ import annotations

import pytest
import torch

from bit_weight_only_q4_gb300 import q4
from tests.test_gpu_prompt_attention import check, made, spans_of

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 2), (6, 2)])
@pytest.mark.parametrize("first", [1, 5, 63, 64, 130, 300])
def test_rows_of_no_score_above_minus_infinity(first, Hq, H, D):
    """The first keys of a sequence give -inf to all: rows that see no others are NaN, as their softmax is, and
    what comes behind them is the attention over the keys that are left."""
    q, k, v, offsets = made([70, 400, 333], Hq, H, D)
    q, k = q.contiguous(), k.contiguous()
    q[:, :, 3] = q[:, :, 3].abs() + 0.25
    lo, hi = 70, 470
    k[lo:lo + first, :, 3] = -INF
    got = q4.q4_prompt_attention(q, k, v, offsets)
    assert got[lo:lo + first].isnan().all()
    check(got, q, k, v, [(0, 70), (lo + first, hi), (470, 803)])
    # of one head of keys alone, and of a whole sequence
    q, k, v, offsets = made([70, 400, 333], Hq, H, D)
    q, k = q.contiguous(), k.contiguous()
    q[:, :, 3] = q[:, :, 3].abs() + 0.25
    k[:70, H - 1, 3] = -INF
    got = q4.q4_prompt_attention(q, k, v, offsets)
    G = Hq // H
    assert got[:70, (H - 1) * G:].isnan().all()
    k[:70, H - 1, 3] = 0
    clean = q4.q4_prompt_attention(q, k, v, offsets)
    assert torch.equal(got[:, :(H - 1) * G], clean[:, :(H - 1) * G])
    check(got, q, k, v, spans_of(offsets)[1:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 2), (6, 2)])
def test_keys_of_no_weight_anywhere(Hq, H, D):
    """Keys of -inf by ones, in runs from 16 to whole tiles and at tiles' beginnings, where references are taken."""
    m = 900
    q, k, v, offsets = made([m], Hq, H, D)
    q, k = q.contiguous(), k.contiguous()
    q[:, :, 3] = q[:, :, 3].abs() + 0.25
    gen = torch.Generator().manual_seed(9)
    gone = torch.rand(m, generator=gen) < 0.1
    for lo, hi in ((128, 144), (192, 208), (256, 320), (384, 512), (512, 530), (640, 900)):
        gone[lo:hi] = True
    gone[0] = False
    k[gone.cuda(), :, 3] = 0
    scale = D**-0.5
    kk, vv = (t.double().repeat_interleave(Hq // H, 1).transpose(0, 1) for t in (k, v))
    s = q.double().transpose(0, 1) @ kk.transpose(1, 2) * scale
    unseen = torch.ones(m, m, dtype=torch.bool, device="cuda").triu(1) | gone.cuda()
    p = s.masked_fill(unseen, -INF).softmax(-1)
    # (the error allowed for goes by the mean of |v| with these probabilities)
    o, mag = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
    d = 2 * D * 2.0**-24 * scale * q.double().norm(dim=-1, keepdim=True) * k.double().norm(dim=-1).max()
    k[gone.cuda(), :, 3] = -INF
    got = q4.q4_prompt_attention(q, k, v, offsets).double()
    assert ((got - o).abs() <= 2.0**-8 * o.abs() + (2.0**-8 + 2 * d) * mag * 1.01 + 1e-30).all()


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (12, 12, 64), (2, 2, 128)])
@pytest.mark.parametrize("swap,units", [(256, 600), (256, 768), (512, 1100), (16, 2000), (1, 300), (4096, 700)])
def test_units_behind_blocks_without_one(swap, units, Hq, H, D):
    """Blocks that have not begun are taken over in an order of the GPU's own: those without work are passed over.  Here
    they come in front of the last `units` % (2 swap) units, up to a swap's length, with every SM busy."""
    gen = torch.Generator().manual_seed(units)
    per = 256 * H // Hq                                      # tokens of a unit
    lens = torch.randint(1, per + 1, (units // H,), generator=gen).tolist()
    q, k, v, offsets = made(lens, Hq, H, D)
    want = q4.q4_prompt_attention(q, k, v, offsets)
    out = torch.full_like(want, 7.0)
    q4.load().q4_test_prompt_swap(swap)
    try:
        for _ in range(3):
            out.fill_(7.0)
            q4.q4_prompt_attention(q, k, v, offsets, out=out)
            assert torch.equal(out, want)
    finally:
        q4.load().q4_test_prompt_swap(0)
    check(want, q, k, v, spans_of(offsets))
    assert q4.device_error_flags() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_large_values_behind_a_low_reference(D):
    """The first reference is 13.9 below (of 2) all scores but its own 16: sums as large as they come, and V of 2^80."""
    m = 33000
    q, k = torch.zeros(m, 1, D, device="cuda"), torch.zeros(m, 1, D, device="cuda")
    q[:, 0, 0] = 1
    k[:, 0, 0] = 13.875
    last = (m - 1) // 128 * 128
    k[last:last + 16, 0, 0] = 0
    gen = torch.Generator("cuda").manual_seed(1)
    v = 2.0**80 * (0.5 + 0.5 * torch.rand(m, 1, D, device="cuda", generator=gen))
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    offsets = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    got = q4.q4_prompt_attention(q, k, v, offsets, scale=0.6931471805599453)
    # rows of the last tile see all keys before it and those up to their own
    p = torch.exp2(k[:, 0, 0].double())
    for r in (last + 20, last + 63, m - 1):
        want = (p[:r + 1, None] * v[:r + 1, 0].double()).sum(0) / p[:r + 1].sum()
        assert ((got[r, 0].double() - want).abs() <= 2 * 2.0**-8 * 1.01 * want).all()
    assert got[last:].isfinite().all()
