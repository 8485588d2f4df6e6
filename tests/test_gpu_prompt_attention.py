"""Causal attention over packed prompts (q4_prompt_attention) against 64 bits.

Errors: the result and the probabilities are each rounded to bf16 (2^-8 of the value, 2^-8 of the weighted
mean of |v|).  Scores are sums of D products in fp32: 2^-24 a step for the D steps of a sum of |q||k| at
most, and as much again for the exponential's argument; a score off by d changes a probability by d of
its value, twice over with the sum it is divided by.
"""
from __future__ import annotations

import math

import pytest
import torch

from bit_weight_only_q4_gb300 import q4

pytestmark = pytest.mark.gpu


def made(lens, Hq, H, D, seed=0, gap=0, strong=2.0):
    """q, k, v as columns of one row, offsets; `gap` rows of no sequence in front and behind."""
    gen = torch.Generator("cuda").manual_seed(seed)
    n = sum(lens) + 2 * gap
    x = torch.randn(n, Hq + 2 * H, D, device="cuda", generator=gen)
    x[:, :Hq] *= strong
    x = x.bfloat16()
    at = [gap]
    for m in lens:
        at.append(at[-1] + m)
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], torch.tensor(at, dtype=torch.int32, device="cuda")


def want(q, k, v, spans, scale):
    """(result, error allowed) in fp64, for the rows of the spans (zeros elsewhere)."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(N, Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for lo, hi in spans:
        kk, vv = (t[lo:hi].double().repeat_interleave(G, 1).transpose(0, 1) for t in (k, v))       # [Hq, m, D]
        for t in range(lo, hi, 512):
            end = min(hi, t + 512)
            qq = q[t:end].double().transpose(0, 1)
            s = qq @ kk[:, :end - lo].transpose(1, 2) * scale
            later = torch.arange(end - lo, device="cuda") > torch.arange(t - lo, end - lo, device="cuda").view(-1, 1)
            s = s.masked_fill(later, -math.inf)
            p = torch.softmax(s, -1)
            o, mag = p @ vv[:, :end - lo], p @ vv[:, :end - lo].abs()
            d = 2 * D * 2.0**-24 * abs(scale) * qq.norm(dim=-1, keepdim=True) * kk.norm(dim=-1).amax(-1).view(-1, 1, 1)
            out[t:end] = o.transpose(0, 1)
            tol[t:end] = (2.0**-8 * o.abs() + (2.0**-8 + 2 * d) * mag * 1.01 + 1e-30).transpose(0, 1)
    return out, tol


def check(got, q, k, v, spans, scale=None):
    ref, tol = want(q, k, v, spans, q.shape[2]**-0.5 if scale is None else scale)
    for lo, hi in spans:
        err = (got[lo:hi].double() - ref[lo:hi]).abs()
        assert (err <= tol[lo:hi]).all(), (lo, hi, float(err.max()), float((err / tol[lo:hi]).max()))


def spans_of(offsets):
    o = offsets.tolist()
    return list(zip(o, o[1:]))


LENGTHS = [[1], [2, 1, 5], [64], [127], [128], [129], [255, 256, 257], [1, 300, 0, 33, 0, 0, 130], [500, 3], [1025]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 1), (6, 2), (8, 2), (12, 12), (28, 4)])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_lengths_and_groups(lens, Hq, H, D):
    q, k, v, offsets = made(lens, Hq, H, D)
    got = q4.q4_prompt_attention(q, k, v, offsets)
    check(got, q, k, v, spans_of(offsets))


@pytest.mark.parametrize("Hq,H,D", [(128, 1, 64), (71, 1, 128), (40, 2, 64), (9, 9, 128), (65, 1, 128)])
def test_other_groups(Hq, H, D):
    q, k, v, offsets = made([131, 1, 70], Hq, H, D)
    check(q4.q4_prompt_attention(q, k, v, offsets), q, k, v, spans_of(offsets))


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (2, 2, 64)])
def test_long_prompts(Hq, H, D):
    q, k, v, offsets = made([4500, 9, 2049], Hq, H, D)
    check(q4.q4_prompt_attention(q, k, v, offsets), q, k, v, spans_of(offsets))


def test_many_sequences():
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (700,), generator=gen).tolist()
    q, k, v, offsets = made(lens, 4, 2, 64)
    check(q4.q4_prompt_attention(q, k, v, offsets), q, k, v, spans_of(offsets))


@pytest.mark.parametrize("Hq,H,D", [(20, 4, 128), (12, 12, 64), (6, 6, 128), (30, 10, 64)])
def test_units_of_every_kind_in_turn(Hq, H, D):
    """Several units for each CTA: pairs of tiles, tiles without a partner, one and many tiles of keys."""
    gen = torch.Generator().manual_seed(5)
    lens = [int(2 ** (11 * x)) for x in torch.rand(60, generator=gen).tolist()]
    q, k, v, offsets = made(lens, Hq, H, D)
    check(q4.q4_prompt_attention(q, k, v, offsets), q, k, v, spans_of(offsets))


def test_rows_of_no_sequence_are_left_alone():
    q, k, v, offsets = made([70, 3, 200], 4, 2, 128, gap=37)
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    got = q4.q4_prompt_attention(q, k, v, offsets, out=out)
    assert got is out
    check(got, q, k, v, spans_of(offsets))
    assert (out[:37] == 7).all() and (out[-37:] == 7).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
def test_scales(scale):
    """Scores of one size to scores in the hundreds, where a reference taken early is far off."""
    q, k, v, offsets = made([700, 100], 4, 2, 64)
    check(q4.q4_prompt_attention(q, k, v, offsets, scale=scale), q, k, v, spans_of(offsets), scale)


def test_scores_that_rise_towards_the_first_key():
    """Tiles are taken from the last to the first: here each holds larger scores than all before it."""
    m, D = 1500, 128
    q, k, v, offsets = made([m], 2, 1, D)
    k = k.contiguous()
    up = torch.linspace(60.0, 0.0, m, device="cuda").view(-1, 1)
    q = torch.zeros_like(q)
    q[:, :, 0] = 1.0
    k[:, :, 0] = up
    for scale in (1.0, 8.0, -1.0, -8.0):
        check(q4.q4_prompt_attention(q, k, v, offsets, scale=scale), q, k, v, spans_of(offsets), scale)


def test_large_and_small_values():
    q, k, v, offsets = made([300], 2, 1, 64)
    v = v.contiguous()
    v[:, :, :32] *= 1e30
    v[:, :, 32:] *= 1e-30
    check(q4.q4_prompt_attention(q, k, v, offsets), q, k, v, spans_of(offsets))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_reaches_only_rows_that_see_it(bad, Hq, H, D):
    lens = [150, 333, 20]
    q, k, v, offsets = made(lens, Hq, H, D)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    clean = q4.q4_prompt_attention(q, k, v, offsets)
    G, spans = Hq // H, spans_of(offsets)
    # in V: one column of the rows that see it, whatever tile it lies in
    for at in (150 + 200, 150 + 0, 150 + 332, 149):
        vb = v.clone()
        vb[at, 0, 5] = bad
        got = q4.q4_prompt_attention(q, k, vb, offsets)
        hit = torch.zeros_like(got, dtype=torch.bool)
        hi = next(h for lo, h in spans if lo <= at < h)
        hit[at:hi, :G, 5] = True
        assert not got[hit].isfinite().any()
        check(torch.where(hit, clean, got), q, k, v, spans)
    # in K: every column of the rows that see it (a key of -inf may leave them finite: it gets no weight)
    kb = k.clone()
    kb[150 + 140, H - 1, 3] = float("nan")
    got = q4.q4_prompt_attention(q, kb, v, offsets)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[290:483, (H - 1) * G:] = True
    assert got[hit].isnan().all()
    check(torch.where(hit, clean, got), q, k, v, spans)
    # in q: its own row
    qb = q.clone()
    qb[160, 1, 0] = float("nan")
    got = q4.q4_prompt_attention(qb, k, v, offsets)
    assert got[160, 1].isnan().all()
    got[160, 1] = clean[160, 1]
    check(got, q, k, v, spans)


def test_rows_around_the_sequences_may_hold_anything():
    q, k, v, offsets = made([70, 200], 4, 2, 128, gap=50)
    clean = q4.q4_prompt_attention(q, k, v, offsets)
    for t in (q, k, v):
        t[:50], t[-50:] = float("nan"), float("inf")
    got = q4.q4_prompt_attention(q, k, v, offsets)
    check(got, q, k, v, spans_of(offsets))
    assert (got[50:-50].double() - clean[50:-50].double()).abs().max() < 0.1


def test_offsets_that_are_not_rising():
    q, k, v, _ = made([200], 2, 1, 64)
    out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    q4.device_error_flags()
    o = torch.tensor([0, 50, 20, 90, 120, 120, 500], dtype=torch.int32, device="cuda")
    q4.q4_prompt_attention(q, k, v, o, out=out)
    assert q4.device_error_flags() == 4
    check(out, q, k, v, [(0, 50), (90, 120), (120, 200)])
    assert (out[50:90] == 7).all()
    q4.q4_prompt_attention(q, k, v, torch.tensor([-5, 60], dtype=torch.int32, device="cuda"), out=out)
    assert q4.device_error_flags() == 4
    check(out, q, k, v, [(0, 60)])


def test_the_same_call_gives_the_same_bits():
    q, k, v, offsets = made([900, 1300, 77], 8, 2, 128)
    a = q4.q4_prompt_attention(q, k, v, offsets)
    for _ in range(5):
        assert torch.equal(q4.q4_prompt_attention(q, k, v, offsets), a)


def test_streams_and_graphs():
    q, k, v, offsets = made([400, 300], 8, 2, 128)
    a = q4.q4_prompt_attention(q, k, v, offsets)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    b = q4.q4_prompt_attention(q, k, v, offsets, stream=side)
    c = q4.q4_prompt_attention(q, k, v, offsets, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = q4.q4_prompt_attention(q, k, v, offsets)
    offsets.copy_(torch.tensor([0, 123, 700], dtype=torch.int32))
    graph.replay()
    check(d, q, k, v, [(0, 123), (123, 700)])
    flags = q4.get_launch_flags()
    q4.set_launch_flags(q4.FLAG_PDL)
    try:
        e = [q4.q4_prompt_attention(q, k, v, offsets) for _ in range(3)]
    finally:
        q4.set_launch_flags(flags)
    assert all(torch.equal(x, d) for x in e)


def test_refusals():
    q, k, v, offsets = made([40], 4, 2, 64)
    for change in (dict(q=q[0]), dict(k=k[:20]), dict(v=v[:, :1]), dict(offsets=offsets.long()), dict(offsets=offsets.cpu()),
                   dict(offsets=offsets[:0]), dict(q=q.float()), dict(k=k.cpu()), dict(out=torch.empty_like(q.contiguous())[:20]),
                   dict(q=q.transpose(0, 1)), dict(v=made([40], 4, 2, 128)[2])):
        args = dict(q=q, k=k, v=v, offsets=offsets)
        args.update(change)
        with pytest.raises(ValueError):
            q4.q4_prompt_attention(**args)
    for change in (dict(scale=float("nan")), dict(q=made([40], 3, 2, 64)[0]),
                   dict(q=made([40], 258, 2, 64)[0])):
        args = dict(q=q, k=k, v=v, offsets=offsets)
        args.update(change)
        with pytest.raises(q4.Q4Error):
            q4.q4_prompt_attention(**args)
    assert q4.q4_prompt_attention(q[:0], k[:0], v[:0], offsets).shape == (0, 4, 64)
    assert q4.device_error_flags() == 0
