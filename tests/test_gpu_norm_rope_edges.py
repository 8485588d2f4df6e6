"""Norms and rotation (q4_norm_rope) where a frequency, a position, a row or eps is at the end of its range."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_weight_only_q4_gb300 import q4
from tests.test_gpu_norm_rope import check, made, want

pytestmark = pytest.mark.gpu


def ints(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("interleaved", [False, True])
def test_negative_frequencies_and_those_next_to_zero(interleaved):
    """Below 2^-52 of a turn and negative: u = f / 2 pi mod 1 lies next to 1, not at -2^-32."""
    f = torch.tensor([-1e-16, -3e-16, -3.6e-16, -1e-12, -1e-30, -0.0, 1e-16, -1.0], device="cuda")
    pos = ints(1, 164, 165, 100003, 1 << 24, (1 << 31) - 1, -(1 << 31), -164)
    q = made(len(pos), 3, 64, 1)
    a, _ = q4.q4_norm_rope(q, None, None, None, pos, f, interleaved=interleaved)
    check(a, q, None, pos, f, interleaved)
    backward, _ = q4.q4_norm_rope(q[:-2], None, None, None, -pos[:-2], -f, interleaved=interleaved)
    check(backward, q[:-2], None, -pos[:-2], -f, interleaved)


PI = 314159265358979323846264338327950288419716939937510582097494459230781640628620899
ONE = 10**80                                                 # (PI is pi * ONE)

# frequency, position whose angle is within 2^-20 of whole turns: there bf16 shows the angle's own error
NEAR_WHOLE_TURNS = [(0.9395782351493835, 2115895823), (0.967883825302124, 2138359862), (0.9996047019958496, 2122168943),
                    (0.9511218070983887, 2127590030), (0.909855306148529, 2136313893), (0.9218469262123108, 2134484148),
                    (0.914912223815918, 2140090169), (0.9124369621276855, 2132787872), (0.9825876951217651, 2134200106),
                    (0.9074194431304932, 2121397446), (0.9759150147438049, 2130958333), (0.9897416234016418, 2114039147)]


def angle(f, p):
    """f p minus the nearest whole turns, by whole numbers; f is a fp32 value."""
    num, den = float(f).as_integer_ratio()
    turn = 2 * PI * den
    rest = num * p * ONE % turn
    return (rest if 2 * rest < turn else rest - turn) / (den * ONE)


@pytest.mark.parametrize("sign", [1, -1])
def test_angles_far_out_are_right_to_2_to_minus_22(sign):
    """Pairs (0, 1) give (-sin, cos); the sine is rounded once, to 2^-8 of itself."""
    n = len(NEAR_WHOLE_TURNS)
    f = torch.tensor([sign * f for f, _ in NEAR_WHOLE_TURNS] + [0.0] * (16 - n), device="cuda")
    pos = ints(*[p for _, p in NEAR_WHOLE_TURNS])
    x = torch.zeros(n, 1, 64, device="cuda", dtype=torch.bfloat16)
    x[:, :, 16:32] = 1
    y, _ = q4.q4_norm_rope(x, None, None, None, pos, f)
    for i, (freq, p) in enumerate(NEAR_WHOLE_TURNS):
        want = angle(sign * freq, p)
        assert abs(want) < 2.0**-19
        assert abs(-float(y[i, 0, i]) - want) <= 2.0**-22 + 2.0**-8 * abs(want), (freq, p)
        assert float(y[i, 0, 16 + i]) == 1


def test_frequencies_above_one():
    """Up to 256 radians a position: whole turns go away exactly."""
    import math

    f = torch.tensor([1.5, 3.1415927, 10.0, 100.3, 255.9, -7.7, 64.0, 128.5], device="cuda")
    pos = ints(0, 1, 77, 65537, (1 << 31) - 1, -(1 << 31), 2123456789, -1999999999)
    x = torch.zeros(len(pos), 1, 64, device="cuda", dtype=torch.bfloat16)
    x[:, :, 8:16] = 1
    y, _ = q4.q4_norm_rope(x, None, None, None, pos, f)
    for i, p in enumerate(pos.tolist()):
        for j, freq in enumerate(f.tolist()):
            a = angle(freq, p)
            # the angle's error, sincospif's (a step of fp32) and the result's rounding
            for got, want in ((-y[i, 0, j], math.sin(a)), (y[i, 0, 8 + j], math.cos(a))):
                assert abs(float(got) - want) <= 2.0**-22 + 2.0**-24 + 2.0**-8 * abs(want), (freq, p)


def check_small(got, x, w, positions, inv_freq, interleaved, eps):
    """As check, and what fp32 loses below 2^-126: a value times its factor, and its partner's added, are each off by
    half of the smallest step, 2^-150, however small they are, before the norm r = 1 / sqrt(mean(x^2) + eps)
    multiplies them: 2^-149 r (without a norm r is 1)."""
    ref, mag = want(x, w, positions, inv_freq, interleaved, eps)
    z = x.double().cpu().numpy()
    r = 1.0 if w is None else 1 / np.sqrt(np.mean(z * z, -1, keepdims=True) + eps)
    assert (np.abs(got.double().cpu().numpy() - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-19 * mag + 2.0**-149 * r + 1e-40).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-30, 2e-22, 2.2e-22, 1e-20, 1e-6])
def test_rows_of_small_values_beside_every_eps(D, eps):
    """Squares that fp32 has few or no digits for: results go by the formula with and without an eps of their size."""
    low = 2.0**-133                                          # bf16's smallest
    sizes = [low, 3 * low, 2.0**-126, 1e-36, 1e-30, 1e-25, 1e-23, 1e-22, 3e-21, 1e-20, 2.0**-49, 2.0**-48, 1e-14, 1e-10, 1.0]
    x = made(len(sizes), 2, D, 5).float()
    x = (x / x.abs().amax(-1, keepdim=True)).double() * torch.tensor(sizes, device="cuda").double().view(-1, 1, 1)
    x = x.bfloat16()
    assert (x.abs().amax((1, 2)) > 0).all()
    w = (1 + 0.25 * torch.arange(D, device="cuda") / D).bfloat16()
    f, pos = 10000.0 ** (-torch.arange(0, 16, device="cuda").float() / 16), torch.arange(len(sizes), device="cuda").int()
    for interleaved in (False, True):
        for k, p, fr in ((w, pos, f), (w, None, None)):
            y, z = q4.q4_norm_rope(x, x, k, None, p, fr, eps=eps, interleaved=interleaved)
            check_small(y, x, k, p, fr, interleaved, float(torch.tensor(eps).float()))
            check_small(z, x, None, p, fr, interleaved, 0.0)


def test_rows_of_every_size_without_an_eps():
    D, top = 64, float(torch.finfo(torch.bfloat16).max)
    x = made(6, 1, D)
    x[0] = x[0].sign() * top
    x[1] = x[1] * 1e-36
    x[2] = x[2] * 1e30
    x[3, 0, 1:] = 0                                          # a single value
    x[3, 0, 0] = 1e25
    x[4, 0, 1:] = 0
    x[4, 0, 0] = 1e-39
    w = (1 + 0.25 * torch.arange(D, device="cuda") / D).bfloat16()
    a, _ = q4.q4_norm_rope(x, None, w, None, None, None, eps=0.0)
    check(a, x, w, None, None, False, eps=0.0)
    x[5] = 0                                                 # 0 / 0
    a, _ = q4.q4_norm_rope(x, None, w, None, None, None, eps=0.0)
    assert a[5].isnan().all()
    check(a[:5], x[:5], w, None, None, False, eps=0.0)


@pytest.mark.parametrize("eps", [1e10, 1e30])
def test_rows_beside_large_eps(eps):
    """To the largest eps that is taken: rows whose squares overflow fp32 and rows that are nothing beside it."""
    top = float(torch.finfo(torch.bfloat16).max)
    sizes = [top, 1e20, 2e19, 1.9e18, 1e16, 1e15, 1e5, 1.0, 1e-10]
    x = made(len(sizes), 2, 128, 6)
    x = (x / x.abs().amax(-1, keepdim=True)).double() * torch.tensor(sizes, device="cuda").double().view(-1, 1, 1)
    x = x.bfloat16()
    w = (1 + 0.25 * torch.arange(128, device="cuda") / 128).bfloat16()
    f, pos = 10000.0 ** (-torch.arange(0, 64, device="cuda").float() / 64), torch.arange(len(sizes), device="cuda").int()
    y, _ = q4.q4_norm_rope(x, None, w, None, pos, f, eps=eps)
    check(y, x, w, pos, f, False, eps=float(torch.tensor(eps).float()))


@pytest.mark.parametrize("D", [64, 128])
def test_an_eps_where_rows_cease_to_be_made_larger(D):
    """2^-72 and 2^-73 and the values next to them, beside sums of squares around 2^-90."""
    sizes = [2.0**-48 * f for f in (0.25, 0.5, 0.68, 0.7, 0.71, 0.98, 0.99, 1.0, 1.01, 1.4)]
    x = made(len(sizes), 2, D, 7).sign().float() * torch.tensor(sizes, device="cuda").view(-1, 1, 1)
    x = x.bfloat16()
    w = (1 + 0.25 * torch.arange(D, device="cuda") / D).bfloat16()
    for top in (2.0**-72, 2.0**-73):
        for eps in (top * (1 - 2.0**-24), top, top * (1 + 2.0**-23)):
            y, _ = q4.q4_norm_rope(x, None, w, None, None, None, eps=eps)
            check(y, x, w, None, None, False, eps=eps)


@pytest.mark.parametrize("top", [2e19, 1e20, 1e30, 3.38e38])
def test_small_values_beside_those_whose_squares_overflow(top):
    """One pair of a row so large that its squares leave fp32's range: the others' results are bf16 numbers still, from
    normal ones down to none."""
    D, n = 128, 40
    x = made(n, 2, D, 8).float()
    x = x / x.abs().amax(-1, keepdim=True) * 2.0 ** -torch.arange(0, 2 * n, 2, device="cuda").view(-1, 1, 1)
    x[:, :, 7] = top
    x[:, :, 64 + 7] = -0.7 * top
    x = x.bfloat16()
    w = (1 + 0.25 * torch.arange(D, device="cuda") / D).bfloat16()
    f, pos = 10000.0 ** (-torch.arange(0, 64, device="cuda").float() / 64), torch.arange(n, device="cuda").int()
    for p, fr in ((pos, f), (None, None)):
        y, _ = q4.q4_norm_rope(x, None, w, None, p, fr, eps=1e-6)
        check_small(y, x, w, p, fr, False, 1e-6)
