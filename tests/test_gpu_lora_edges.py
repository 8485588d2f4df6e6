"""Adapters of many requests (q4_lora): what each of its kernels reports, and its sums' width.

FEW, SHARED and MANY are calls that go to the kernel of a request's few tokens, of requests that share adapters, and
of many tokens: (tokens of each request, adapters).
"""
from __future__ import annotations

import pytest
import torch

from bit_weight_only_q4_gb300 import q4
from tests.test_gpu_lora import Case

pytestmark = pytest.mark.gpu

FEW, SHARED, MANY = ([1] * 64, 128), ([1] * 64, 8), ([40] * 64, 8)
KERNELS = pytest.mark.parametrize("lens,adapters", [FEW, SHARED, MANY], ids=["few", "shared", "many"])


def with_empty_requests(lens, adapters, empty):
    """The requests and `empty` more, of no tokens, behind them."""
    ids = [b % adapters for b in range(len(lens))]
    return Case(lens + [0] * empty, ids + [0] * empty, 128, 256, 16, adapters=adapters)


@KERNELS
@pytest.mark.parametrize("at", [64, 70, 100, 127])
@pytest.mark.parametrize("value", [3, -1, 1 << 20])
def test_offsets_behind_the_last_token_are_looked_at(lens, adapters, at, value):
    """Requests 64 .. 127 have no tokens; an offset among theirs that falls or lies outside is reported all the same."""
    case = with_empty_requests(lens, adapters, 64)
    q4.device_error_flags()
    ref = case()
    assert q4.device_error_flags() == 0
    case.check(ref)
    o = case.offsets.clone()
    o[at + 1] = value
    got = case(offsets=o)
    assert q4.device_error_flags() == 4
    assert torch.equal(got, ref)


@KERNELS
@pytest.mark.parametrize("at", [0, 5, 40, 64, 100, 127])
def test_ids_of_requests_without_tokens_are_looked_at(lens, adapters, at):
    """An id past the adapters is reported whether its request has tokens or not, and whichever kernel runs."""
    if at < 64:
        lens = lens[:at] + [0] + lens[at + 1:]
    case = with_empty_requests(lens, adapters, 64)
    q4.device_error_flags()
    ref = case()
    assert q4.device_error_flags() == 0
    case.check(ref)
    ids = case.ids.clone()
    ids[at] = adapters
    got = case(ids=ids)
    assert q4.device_error_flags() == 4
    assert torch.equal(got, ref)
    ids[at] = -7
    assert torch.equal(case(ids=ids), ref) and q4.device_error_flags() == 0


@pytest.mark.parametrize("N", [8, 56, 64, 72, 1000, 2048, 23000])
@pytest.mark.parametrize("lens", [[1] * 9, [3, 8, 0, 2] * 20, [300, 1, 0, 33, 128], [128] * 40], ids=["one", "few", "many", "tiles"])
def test_requests_without_an_adapter(lens, N):
    """base as it is, from shares of no columns to shares of more than a CTA has threads, and no row beside theirs."""
    for adapters in (1, 200):
        case = Case(lens, [-1] * len(lens), 64, N, 8, adapters=adapters, gap=3)
        out = torch.full_like(case.base, 5.0)
        case(out=out)
        assert torch.equal(out[3:-3], case.base[3:-3]) and (out[:3] == 5).all() and (out[-3:] == 5).all()


@pytest.mark.parametrize("rank", [8, 16, 40, 64, 72, 128])
@pytest.mark.parametrize("K", [64, 136])
@pytest.mark.parametrize("lens,adapters", [FEW, SHARED, ([3, 8, 0, 1, 5] * 9, 45), ([3, 8, 0, 1, 5] * 9, 3)],
                         ids=["few", "shared", "few drafts", "shared drafts"])
def test_sums_between_the_products_of_few_tokens_have_twice_the_digits(lens, adapters, K, rank):
    """t = x A^T meets B as two bf16 values, each off by 2^-8 of what it stands for: 2^-16 of t is left.  Beside it
    there are fp32's steps, 2^-23 each (the tensor cores cut), for K + 2 rank products and 32 sums of parts, and the result's
    rounding.  With base 0, t as one bf16 value would be outside that."""
    case = Case(lens, [b % adapters for b in range(len(lens))], K, 1024, rank, adapters=adapters)
    case.base.zero_()
    got = case()
    beyond = 0
    for lo, hi, i in zip(case.at, case.at[1:], case.id_list):
        x, a, b, s = case.x[lo:hi].double(), case.a[i].double(), case.b[i].double(), case.scales[i].double()
        t = x @ a.T
        want = s * (t @ b.T)
        sums = s * ((x.abs() @ a.abs().T) @ b.abs().T)
        tol = 1.01 * (2.0**-8 * want.abs() + 2.0**-16 * s * (t.abs() @ b.abs().T) + 2.0**-23 * (K + 2 * rank + 32) * sums)
        assert ((got[lo:hi].double() - want).abs() <= tol).all()
        once = (s * (t.bfloat16().double() @ b.T)).bfloat16().double()
        beyond += int(((once - want).abs() > tol).sum())
    assert beyond > 0
