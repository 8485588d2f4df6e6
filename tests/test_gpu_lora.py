"""Adapters of many requests beside a projection (q4_lora) against 64 bits.

Errors: the result and x A^T are each rounded to bf16 (2^-8 of the value, 2^-8 of the sum of |t b|), and the two
sums are fp32: a step of 2^-24 for each of their K and rank terms, of the sums of the terms' magnitudes.
"""
from __future__ import annotations

import pytest
import torch

from bit_weight_only_q4_gb300 import q4

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, ids, K, N, rank, adapters=None, seed=0, gap=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        n, count = sum(lens) + 2 * gap, adapters or max(max(ids) + 1, 1)
        at = [gap]
        for m in lens:
            at.append(at[-1] + m)
        self.lens, self.id_list, self.at = lens, ids, at
        self.x, self.base = rand(n, K).bfloat16(), rand(n, N).bfloat16()
        self.a, self.b = (rand(count, rank, K) * K**-0.5).bfloat16(), (rand(count, N, rank) * rank**-0.5).bfloat16()
        self.scales = 0.25 + 1.75 * torch.rand(count, device="cuda", generator=gen)
        self.offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")

    def __call__(self, **change):
        args = dict(x=self.x, a=self.a, b=self.b, scales=self.scales, offsets=self.offsets, ids=self.ids, base=self.base)
        args.update(change)
        return q4.q4_lora(**args)

    def want(self, x=None, base=None):
        """(result, error allowed) in fp64; rows of no request as base."""
        x, out = (self.x if x is None else x).double(), (self.base if base is None else base).double().clone()
        tol = torch.zeros_like(out)
        K, r = self.a.shape[2], self.a.shape[1]
        for lo, hi, i in zip(self.at, self.at[1:], self.id_list):
            if i >= 0:
                a, b, s = self.a[i].double(), self.b[i].double(), self.scales[i].double()
                t = x[lo:hi] @ a.T
                sums = (x[lo:hi].abs() @ a.abs().T) @ b.abs().T
                out[lo:hi] += s * (t @ b.T)
                tol[lo:hi] = 2.0**-8 * out[lo:hi].abs() + s * (2.0**-8 * (t.abs() @ b.abs().T) + 2.0**-24 * (K + r) * sums)
        return out, tol * 1.01

    def check(self, got, rows=None, **change):
        ref, tol = self.want(**change)
        rows = slice(self.at[0], self.at[-1]) if rows is None else rows
        err = (got[rows].double() - ref[rows]).abs()
        assert (err <= tol[rows]).all(), (float(err.max()), float((err / tol[rows].clamp(min=1e-30)).max()))


FEW = [([1], [0]), ([1] * 48, list(range(48))), ([5] * 20, [b % 3 for b in range(20)]), ([8, 0, 1, 3, 0, 7], [1, 0, -1, 0, 2, 2]),
       ([40] + [1] * 30, [0] + [b % 5 for b in range(30)])]
MANY = [([9], [0]), ([128], [0]), ([127, 129], [1, 0]), ([300, 1, 0, 33, 70], [0, 1, 1, -1, 2]), ([1000, 31, 32, 64], [1, 0, 1, 0]),
        ([17] * 9, [b % 4 for b in range(9)])]


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 48, 64, 72, 104, 128])
@pytest.mark.parametrize("lens,ids", FEW + MANY, ids=str)
def test_requests_and_ranks(lens, ids, rank):
    case = Case(lens, ids, 512, 1024, rank)
    case.check(case())


@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("tiles", [1, 41, 48, 58, 70, 90, 120, 160])
def test_clusters_of_every_size(tiles, rank):
    """From eight CTAs for a tile to two, as tiles become more; pieces of K and N that do not share out evenly."""
    lens = [128 * (tiles // 2) + 100, 0, 128 * (tiles - tiles // 2) - 128 + 61]
    case = Case(lens, [1, 0, 0], 328, 840, rank)
    case.check(case())


@pytest.mark.parametrize("rank", [8, 16, 40, 64, 72, 128])
@pytest.mark.parametrize("spare", [0, 200])
def test_requests_that_share_adapters_and_adapters_to_spare(spare, rank):
    """Few tokens each: tiles by adapter where requests share them, and by request where there are as many adapters."""
    gen = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 9, (200,), generator=gen).tolist()
    ids = torch.randint(-1, 6, (200,), generator=gen).tolist()
    case = Case(lens, ids, 264, 392, rank, adapters=6 + spare, gap=5)
    out = torch.full_like(case.base, 5.0)
    case.check(case(out=out))
    assert (out[:5] == 5).all() and (out[-5:] == 5).all()
    got = case(base=(base := case.base.clone()), out=base)
    assert torch.equal(got[5:-5], out[5:-5]) and torch.equal(got[:5], case.base[:5]) and torch.equal(got[-5:], case.base[-5:])
    # one adapter for all, and none for any
    for ids in ([3] * 200, [-1] * 200):
        case.id_list = ids
        case.check(case(ids=torch.tensor(ids, dtype=torch.int32, device="cuda")))


@pytest.mark.parametrize("adapters", [2, 200])
def test_few_tokens_with_offsets_and_ids_that_are_none(adapters):
    q4.device_error_flags()
    case = Case([3] * 40, [b % 2 for b in range(40)], 128, 256, 16, adapters=adapters)
    o = case.offsets.clone()
    o[10], o[20], o[40] = 5, 1000, 118                      # 10 falls back, 20 is past the end, 40 ends early
    ids = case.ids.clone()
    ids[3] = adapters
    out = torch.full_like(case.base, 5.0)
    case(offsets=o, ids=ids, out=out)
    assert q4.device_error_flags() == 4
    # request 9 ends before it begins; 10 begins before 9 in front of it does not end ... what is left is in order
    spans = []
    floor, at = 0, o.tolist()
    for b, (lo, hi) in enumerate(zip(at, at[1:])):
        lo, hi = min(max(lo, 0), 120), min(max(hi, 0), 120)
        if hi >= lo and lo >= floor:
            spans.append((lo, hi, -1 if b == 3 else b % 2))
        floor = max(floor, hi)
    case.at, case.id_list = [0], []
    ref, tol = case.base.double().clone(), torch.full(case.base.shape, 0.0, dtype=torch.float64, device="cuda")
    seen = torch.zeros(120, dtype=torch.bool, device="cuda")
    for lo, hi, i in spans:
        case.at, case.id_list = [lo, hi], [i]
        a, b = case.want()
        ref[lo:hi], tol[lo:hi] = a[lo:hi], b[lo:hi]
        seen[lo:hi] = True
    assert ((out[seen].double() - ref[seen]).abs() <= tol[seen]).all() and (out[~seen] == 5).all()


@pytest.mark.parametrize("K,N", [(8, 8), (16, 520), (72, 8), (136, 264), (1000, 72), (2048, 2048), (8192, 1048), (776, 2584)])
@pytest.mark.parametrize("lens,ids", [FEW[3], MANY[3]], ids=str)
def test_sizes(lens, ids, K, N):
    for rank in (8, 56, 128):
        case = Case(lens, ids, K, N, rank)
        case.check(case())


@pytest.mark.parametrize("lens,ids", [FEW[3], FEW[4], MANY[3], MANY[4]], ids=str)
@pytest.mark.parametrize("N", [200, 2048])
def test_in_place_and_columns_of_wider_rows(lens, ids, N):
    case = Case(lens, ids, 256, N, 16, gap=13)
    ref = case()
    n = case.x.shape[0]
    wide = torch.full((n, N + 72), 7.0, device="cuda", dtype=torch.bfloat16)
    wide[:, 32:32 + N] = case.base
    part = wide[:, 32:32 + N]
    xw = torch.zeros(n, 256 + 40, device="cuda", dtype=torch.bfloat16)
    xw[:, 8:264] = case.x
    got = case(x=xw[:, 8:264], base=part, out=part)
    assert got is part
    assert torch.equal(got[13:-13], ref[13:-13])
    case.check(got)
    assert torch.equal(part[:13], case.base[:13]) and torch.equal(part[-13:], case.base[-13:])
    assert (wide[:, :32] == 7).all() and (wide[:, 32 + N:] == 7).all()
    out = torch.full_like(case.base, 5.0)
    case(out=out)
    assert (out[:13] == 5).all() and (out[-13:] == 5).all() and torch.equal(out[13:-13], ref[13:-13])


@pytest.mark.parametrize("lens,ids", [([1] * 5, [0, -1, 9, 1, 0]), ([100, 200, 50], [0, 7, -1])], ids=str)
def test_ids_past_the_adapters(lens, ids):
    q4.device_error_flags()
    case = Case(lens, [i if i < 5 else -1 for i in ids], 128, 256, 16, adapters=2)
    got = case(ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
    assert q4.device_error_flags() == 4
    case.check(got)


@pytest.mark.parametrize("n", [6, 600])
def test_offsets_that_are_not_rising(n):
    q4.device_error_flags()
    case = Case([n // 3, n // 3, n // 3], [0, 1, 0], 128, 256, 16)
    o = torch.tensor([0, n // 3, 0, n + 50], dtype=torch.int32, device="cuda")
    out = torch.full_like(case.base, 5.0)
    case(offsets=o, out=out)
    assert q4.device_error_flags() == 4
    case.check(out, rows=slice(0, n // 3))
    assert (out[n // 3:] == 5).all()


@pytest.mark.parametrize("lens,ids", [([3, 1, 8], [0, 1, 0]), ([150, 33], [0, 1])], ids=str)
def test_what_is_not_finite_stays_in_its_token(lens, ids):
    for rank in (8, 24, 72):
        case = Case(lens, ids, 256, 512, rank)
        clean = case()
        x = case.x.clone()
        x[2, 17] = float("nan")
        x[lens[0], 3] = float("inf")
        got = case(x=x)
        assert got[2].isnan().all() and not got[lens[0]].isfinite().any()
        got[2], got[lens[0]] = clean[2], clean[lens[0]]
        assert torch.equal(got, clean)
        # another adapter's values, and rows beside a request's, count for nothing
        case.a[1], case.b[1] = float("nan"), float("inf")
        got = case()
        assert torch.equal(got[:lens[0]], clean[:lens[0]])


def test_many_requests():
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 3, (900,), generator=gen).tolist()
    case = Case(lens, torch.randint(-1, 30, (900,), generator=gen).tolist(), 256, 256, 16, adapters=30)
    case.check(case())
    lens = torch.randint(0, 40, (300,), generator=gen).tolist()
    case = Case(lens, torch.randint(-1, 30, (300,), generator=gen).tolist(), 256, 256, 16, adapters=30)
    case.check(case())


@pytest.mark.parametrize("lens,ids", [FEW[1], MANY[4]], ids=str)
def test_streams_graphs_and_the_same_bits(lens, ids):
    case = Case(lens, ids, 1024, 2048, 32)
    ref = case()
    for _ in range(4):
        assert torch.equal(case(), ref)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = case(stream=side), case(stream=other)
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = case()
    case.x.mul_(-1.5)
    case.ids.copy_(case.ids.flip(0))
    case.id_list = case.id_list[::-1]
    graph.replay()
    case.check(out)
    q4.set_launch_flags(q4.FLAG_PDL)
    try:
        chain = [case() for _ in range(3)]
    finally:
        q4.set_launch_flags(0)
    assert all(torch.equal(c, out) for c in chain)


def test_refusals():
    case = Case([3, 4], [0, 1], 64, 128, 16)
    for change in (dict(x=case.x[0]), dict(x=case.x[:, :32]), dict(a=case.a[:1]), dict(b=case.b[:, :, :8]), dict(scales=case.scales[:1]),
                   dict(scales=case.scales.double()), dict(offsets=case.offsets[:2]), dict(offsets=case.offsets.long()),
                   dict(ids=case.ids.long()), dict(base=case.base[:3]), dict(base=case.base.float()), dict(x=case.x.cpu()),
                   dict(out=case.base[:, :64]), dict(a=case.a.transpose(1, 2)), dict(ids=case.ids.cpu()),
                   dict(x=torch.empty(64, 7, device="cuda", dtype=torch.bfloat16).t())):
        with pytest.raises(ValueError):
            case(**change)
    for rank, K, N in ((4, 64, 128), (136, 64, 128), (12, 64, 128), (16, 60, 128), (16, 64, 100)):
        with pytest.raises(q4.Q4Error):
            Case([3, 4], [0, 1], K, N, rank)()
    assert case(x=case.x[:0], base=case.base[:0]).shape == (0, 128)
    assert q4.device_error_flags() == 0
