"""Norms of queries and keys with the position rotation (q4_norm_rope) against 64 bits.

A result is rounded once to bf16 (half a step, 2^-8 of the value).  What is left is fp32: the norm,
the weight and the turn are some ten operations of 2^-24, the angle is right to 2^-22 of a radian:
2^-19 of the pair's length covers both.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_weight_only_q4_gb300 import q4

pytestmark = pytest.mark.gpu
EPS = 1e-6


def want(x, w, positions, inv_freq, interleaved, eps=EPS):
    """(result, length of each value's pair) in fp64 of x [..., heads, D]."""
    y = x.double().cpu().numpy().reshape(-1, x.shape[-2], x.shape[-1])
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps) * w.double().cpu().numpy()
    mag = np.abs(y)
    if positions is not None:
        f = inv_freq.cpu().numpy().astype(np.float64)
        p = positions.cpu().numpy().astype(np.float64)
        turns = np.outer(p, f)                               # exact: 31 + 24 bits
        cos, sin = np.cos(turns)[:, None], np.sin(turns)[:, None]
        i = np.arange(len(f))
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + len(f))
        a, b = y[..., one].copy(), y[..., two].copy()
        y, mag = y.copy(), mag.copy()
        y[..., one], y[..., two] = a * cos - b * sin, b * cos + a * sin
        mag[..., one] = mag[..., two] = np.abs(a) + np.abs(b)
    return y.reshape(x.shape), mag.reshape(x.shape)


def check(got, x, w, positions, inv_freq, interleaved, eps=EPS):
    ref, mag = want(x, w, positions, inv_freq, interleaved, eps)
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-19 * mag + 1e-40).all()


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(0, R, 2).float() / R)).cuda()


def made(tokens, heads, D, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(tokens, heads, D, device="cuda", generator=gen) * torch.exp(
        torch.randn(tokens, 1, 1, device="cuda", generator=gen))
    return x.bfloat16()


def weight(D, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(D, device="cuda", generator=gen)).bfloat16()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (64, 48), (64, 16), (128, 128), (128, 64), (128, 48), (128, 16), (128, 112)])
@pytest.mark.parametrize("tokens,Hq,H", [(1, 1, 1), (5, 7, 1), (33, 16, 16), (301, 5, 3)])
def test_norms_and_rotation(tokens, Hq, H, D, R, interleaved):
    q, k = made(tokens, Hq, D, 1), made(tokens, H, D, 2)
    wq, wk = weight(D, 3), weight(D, 4)
    pos = torch.randint(0, 1 << 20, (tokens,), device="cuda", dtype=torch.int32)
    f = freqs(R)
    a, b = q4.q4_norm_rope(q, k, wq, wk, pos, f, interleaved=interleaved)
    check(a, q, wq, pos, f, interleaved)
    check(b, k, wk, pos, f, interleaved)


def test_many_tokens_of_a_fused_row():
    """Enough tokens for a warp to take several whole ones, q and k as columns of one row, in place."""
    T, Hq, H, D = 5003, 14, 3, 128
    row = made(T, Hq + 2 * H, D)
    keep = row.clone()
    q, k = row[:, :Hq], row[:, Hq:Hq + H]
    wq, wk, f = weight(D, 3), weight(D, 4), freqs(D)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    a, b = q4.q4_norm_rope(q, k, wq, wk, pos, f)
    check(a, q, wq, pos, f, False)
    check(b, k, wk, pos, f, False)
    got = q4.q4_norm_rope(q, k, wq, wk, pos, f, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(row[:, Hq + H:], keep[:, Hq + H:])    # v beside them


def test_layouts_of_the_layer():
    """q as [batch, tokens, heads, D], k as [batch * tokens, heads, D]; results elsewhere, strided."""
    B, T, Hq, H, D = 3, 5, 8, 2, 64
    row = made(B * T, Hq + 2 * H, D)
    q, k = row[:, :Hq].view(B, T, Hq, D), row[:, Hq:Hq + H]
    f, pos = freqs(D), torch.arange(B * T, device="cuda", dtype=torch.int32)
    w = weight(D, 1)
    wide = torch.full((B * T, H + 3, D), 7.0, device="cuda", dtype=torch.bfloat16)
    a, b = q4.q4_norm_rope(q, k, w, None, pos, f, k_out=wide[:, 1:1 + H])
    assert a.shape == q.shape
    check(a, q, w, pos, f, False)
    check(b, k, None, pos, f, False)
    assert (wide[:, 0] == 7).all() and (wide[:, 1 + H:] == 7).all()


@pytest.mark.parametrize("norm", [True, False])
def test_parts_that_are_left_out(norm):
    q, k = made(9, 3, 128), made(9, 2, 128, 1)
    w = weight(128, 1) if norm else None
    a, b = q4.q4_norm_rope(q, k, w, w, None, None)
    check(a, q, w, None, None, False)
    check(b, k, w, None, None, False)
    a, b = q4.q4_norm_rope(q, None, w, None, torch.arange(9, device="cuda", dtype=torch.int32), freqs(64))
    assert b is None
    check(a, q, w, torch.arange(9), freqs(64), False)
    empty = q4.q4_norm_rope(q[:0], k[:0], w, w, None, None)
    assert empty[0].shape == (0, 3, 128) and empty[1].shape == (0, 2, 128)


def test_far_and_negative_positions():
    pos = torch.tensor([0, 1, 4095, 131071, (1 << 24) + 1, (1 << 31) - 1, -1, -77777, -(1 << 31)], dtype=torch.int32,
                       device="cuda")
    q = made(len(pos), 2, 128)
    f = freqs(128)
    a, _ = q4.q4_norm_rope(q, None, None, None, pos, f)
    check(a, q, None, pos, f, False)


def test_rows_of_every_size():
    """Rows of zeros, of the largest and the smallest values: squares leave fp32's range, results do not."""
    D, top = 64, float(torch.finfo(torch.bfloat16).max)
    x = made(6, 1, D)
    x[0] = 0
    x[1] = x[1].sign() * top
    x[2] = x[2] * 1e-36
    x[3] = x[3] * 1e30
    x[4, 0, 1:] = 0                                          # a single value
    x[4, 0, 0] = 1e25
    w = weight(D, 1)
    a, _ = q4.q4_norm_rope(x, None, w, None, None, None)
    check(a, x, w, None, None, False)
    a, _ = q4.q4_norm_rope(x[1:], None, w, None, None, None, eps=0.0)
    check(a[2:], x[3:], w, None, None, False, eps=0.0)


def test_what_is_not_finite_stays_in_its_head():
    q = made(4, 4, 128)
    w, f, pos = weight(128, 1), freqs(128), torch.arange(4, device="cuda", dtype=torch.int32)
    clean, _ = q4.q4_norm_rope(q, None, w, None, pos, f)
    q[1, 2, 5] = float("nan")
    q[2, 1, 70] = float("inf")
    got, _ = q4.q4_norm_rope(q, None, w, None, pos, f)
    assert got[1, 2].isnan().all() and got[2, 1, 70].isnan() and got[2, 1, 6].isnan()
    got[1, 2], got[2, 1] = clean[1, 2], clean[2, 1]
    assert torch.equal(got, clean)


def test_streams_and_graphs():
    q, k = made(48, 16, 128), made(48, 16, 128, 1)
    w, f = weight(128, 1), freqs(128)
    pos = torch.arange(48, device="cuda", dtype=torch.int32)
    want_q, want_k = q4.q4_norm_rope(q, k, w, w, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = q4.q4_norm_rope(q, k, w, w, pos, f, stream=side)
    side.synchronize()
    assert torch.equal(a, want_q) and torch.equal(b, want_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = q4.q4_norm_rope(q, k, w, w, pos, f)
    pos += 1000
    graph.replay()
    want_q, want_k = q4.q4_norm_rope(q, k, w, w, pos, f)
    assert torch.equal(a, want_q) and torch.equal(b, want_k)


def test_refusals():
    q, k, w = made(4, 2, 64), made(4, 1, 64), weight(64, 1)
    pos, f = torch.arange(4, device="cuda", dtype=torch.int32), freqs(64)
    bad = [dict(q=q[0]), dict(k=made(5, 1, 64)), dict(q_weight=w[:32]), dict(q_weight=w.float()), dict(positions=pos.long()),
           dict(positions=pos[:3]), dict(inv_freq=f.double()), dict(positions=None), dict(q=q.float()), dict(q=q.cpu()),
           dict(q_out=made(4, 3, 64)), dict(q=q.transpose(0, 1)), dict(k_weight=w.cpu())]
    for change in bad:
        args = dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, inv_freq=f)
        args.update(change)
        with pytest.raises(ValueError):
            q4.q4_norm_rope(**args)
    for change in (dict(eps=-1.0), dict(eps=float("nan")), dict(inv_freq=f[:20].contiguous()),
                   dict(inv_freq=freqs(128)), dict(q=made(4, 2, 96))):
        args = dict(q=q, k=None, q_weight=None, k_weight=None, positions=pos, inv_freq=f)
        args.update(change)
        with pytest.raises(q4.Q4Error):
            q4.q4_norm_rope(**args)
