"""The paged key/value cache on the GPU against the plain reference of kv_reference.py.

Writing and reading back are exact: every step is one fp32 operation, so the stored
bytes and the bf16 values must match bit for bit.  Attention (fp64 reference on the
same cached values) is held per output element to
    |err| <= 2^-8 |o| + 2^-9 sum_j p_j |v_j| + 2^-126
2^-8 |o| is the bf16 rounding of the output (half an ulp is 2^-9 |o|) with as much
again for its being taken of a perturbed value.  The second term covers what perturbs the sum:
the probabilities times the V scale rounded to fp16 (2^-11 of each term), and scores
off by at most 2^-12 -- fp32 sums of D products, at most 2 D 2^-24 of sum |q k| scale,
which the inputs here keep below 2^4 -- which moves every p_j, and their sum, by as much.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import kv_reference as R

pytestmark = pytest.mark.gpu

FMTS = [R.INT8, R.INT4]


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_weight_only_q4_gb300 import build, q4 as lib
    build.build()
    lib.load()
    lib.set_launch_flags(0)
    return lib


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16()


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def same_bf16(got, want):
    """Bit equality, any NaN equal to any NaN."""
    g, w = got.float().cpu().numpy(), bf16(want).float().numpy()
    nan = np.isnan(w)
    np.testing.assert_array_equal(np.isnan(g), nan)
    np.testing.assert_array_equal(np.where(nan, 0, g), np.where(nan, 0, w))


def rows(rng, n, H, D):
    return bf16(rng.standard_normal((n, H, D))).float().numpy()


def special_rows(rng, n, H, D):
    x = rows(rng, n, H, D)
    kinds = [np.zeros(D), np.full(D, -3.25), np.full(D, 1e-30), np.linspace(-1e-7, 1e-7, D),
             np.linspace(-3e38, 3e38, D), np.linspace(70000, 9e4, D), np.arange(D) - D / 2,
             np.r_[np.inf, np.zeros(D - 1)], np.r_[np.zeros(D - 1), np.nan],
             np.r_[-np.inf, np.ones(D - 1)], np.linspace(2.0**-14, 2.0**-13, D), np.full(D, 65504.0 * 127)]
    for i in range(min(n, len(kinds))):
        x[i, i % H] = kinds[i]
    return bf16(x).float().numpy()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,H,page", [(1, 1, 16), (37, 3, 32), (300, 8, 128)])
def test_write_stores_the_reference_bytes(q4, fmt, D, n, H, page):
    rng = np.random.default_rng([1, fmt, D, n])
    pages = -(-n // page) + 2
    init = rng.integers(0, 256, (pages, H, page // 16, R.block_bytes(fmt, D)), dtype=np.uint8)
    k, v = special_rows(rng, n, H, D), special_rows(rng, n, H, D)[::-1].copy()
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    if n > 2:
        slots[1] = -1
    want = init.copy()
    R.write(want, slots, k, v, fmt, page)
    # K and V as columns of one wider row per token, V first
    wide = torch.zeros(n, 2 * H * D + 24, dtype=torch.bfloat16)
    wide[:, 8:8 + H * D] = bf16(v).view(n, -1)
    wide[:, 16 + H * D:16 + 2 * H * D] = bf16(k).view(n, -1)
    wide = wide.cuda()
    cache = torch.from_numpy(init).cuda()
    q4.device_error_flags(clear=True)
    q4.q4_kv_write(wide[:, 16 + H * D:16 + 2 * H * D].view(n, H, D), wide[:, 8:8 + H * D].view(n, H, D),
                   cache, torch.from_numpy(slots).cuda(), fmt)
    assert q4.device_error_flags() == 0
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_write_of_ties_and_of_rows_of_every_size(q4, fmt, D):
    """Values halfway between two codes, and rows from below fp16's smallest scale to past its
    largest: the bytes of the reference's divisions."""
    rng = np.random.default_rng([15, fmt, D])
    rows_ = []
    for e in range(-40, 36):
        half = rng.integers(-127, 127, D) + 0.5             # int8: ties at a scale of 2^e
        half[:2] = 127, -100
        rows_.append(half * 2.0**e)
        half = rng.integers(0, 15, D) + 0.5 - 7             # int4: the same, from the minimum on
        half[:2] = -7, 8
        rows_.append(half * 2.0**e)
        rows_.append(rng.standard_normal(D) * 2.0**e)
        rows_.append((rng.integers(0, 16, D) - 100) * 2.0**e)                # far from zero
    x = bf16(np.stack(rows_)).float().numpy().reshape(-1, 4, D)
    n, H, page = *x.shape[:2], 16
    init = np.zeros((-(-n // page), H, 1, R.block_bytes(fmt, D)), np.uint8)
    want = init.copy()
    R.write(want, np.arange(n), x, x[::-1].copy(), fmt, page)
    cache = torch.from_numpy(init).cuda()
    q4.q4_kv_write(bf16(x).cuda(), bf16(x[::-1].copy()).cuda(), cache, torch.arange(n, dtype=torch.int32, device="cuda"), fmt)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


def test_write_leaves_out_slots_outside_the_cache(q4):
    rng = np.random.default_rng(2)
    init = rng.integers(0, 256, (2, 2, 1, R.block_bytes(0, 64)), dtype=np.uint8)
    k, v = rows(rng, 4, 2, 64), rows(rng, 4, 2, 64)
    slots = np.array([5, 32, -7, 2**31 - 1], np.int32)
    want = init.copy()
    R.write(want, slots, k, v, 0, 16)
    cache = torch.from_numpy(init).cuda()
    q4.device_error_flags(clear=True)
    q4.q4_kv_write(bf16(k).cuda(), bf16(v).cuda(), cache, torch.from_numpy(slots).cuda(), 0)
    assert q4.device_error_flags() == 4
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


def filled(rng, fmt, D, H, page, lens, extra=1, prefix=0):
    """A cache of random pages: (bytes, table, prefix pages, per-sequence (k, v)) -- every byte that
    no token owns is random (NaN scales among them)."""
    need = [-(-n // page) for n in lens]
    pre = -(-prefix // page)
    total = sum(need) + pre + extra
    cache = rng.integers(0, 256, (total, H, page // 16, R.block_bytes(fmt, D)), dtype=np.uint8)
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    pp = order[at:at + pre]
    for pages, n in [*zip(table, lens), (pp, prefix)]:
        pos = np.arange(n)
        if n:
            slots = pages[pos // page].astype(np.int64) * page + pos % page
            R.write(cache, slots, rows(rng, n, H, D), rows(rng, n, H, D), fmt, page)
    return cache, table, pp


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,page,lens,most", [(1, 16, [1], 1), (3, 32, [0, 33, 100, 64], 100), (8, 64, [129, 5], 200)])
def test_read_returns_the_cached_values(q4, fmt, D, H, page, lens, most):
    rng = np.random.default_rng([3, fmt, D, H])
    cache, table, _ = filled(rng, fmt, D, H, page, lens)
    q4.device_error_flags(clear=True)
    k, v = q4.q4_kv_read(torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(),
                         torch.tensor(lens, dtype=torch.int32, device="cuda"), most, D, fmt)
    assert q4.device_error_flags() == 0
    assert tuple(k.shape) == (len(lens), most, H, D)
    for b, n in enumerate(lens):
        kk, vv, _ = R.read(cache, table[b], n, fmt, D)
        same_bf16(k[b, :n], kk)
        same_bf16(v[b, :n], vv)
        assert not bits(k[b, n:]).any() and not bits(v[b, n:]).any()


def test_read_of_poisoned_rows_and_bad_pages(q4):
    rng = np.random.default_rng(4)
    fmt, D, H, page = 0, 64, 2, 16
    cache, table, _ = filled(rng, fmt, D, H, page, [40, 20])
    bad = rows(rng, 1, H, D)
    bad[0, 1, 3] = np.inf
    slot = int(table[0, 0]) * page + 2
    R.write(cache, [slot], bad, bad, fmt, page)
    table[1, 0] = cache.shape[0]                            # not a page
    q4.device_error_flags(clear=True)
    k, v = q4.q4_kv_read(torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(),
                         torch.tensor([40, 90], dtype=torch.int32, device="cuda"), 90, D, fmt)
    assert q4.device_error_flags() == 4
    kk, vv, _ = R.read(cache, table[0], 40, fmt, D)
    assert np.isnan(kk[2, 1]).all() and not np.isnan(kk[2, 0]).any()
    same_bf16(k[0, :40], kk)
    same_bf16(v[0, :40], vv)
    assert not bits(k[1, :16]).any()                        # the bad page
    assert not bits(k[1, 48:]).any()                        # past the table
    assert bits(k[1, 16:20]).any()


def check(out, q, cache, table, lens, fmt, scale, prefix_pages=(), prefix=0):
    B, T, Hq, D = q.shape
    out = out.float().cpu().numpy().astype(np.float64)
    worst = 0.0
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * cache.shape[2] * 16))
        k, v, ok = R.read(cache, table[b], n, fmt, D)
        if prefix:
            kp, vp, okp = R.read(cache, prefix_pages, prefix, fmt, D)
            k, v, ok = np.concatenate((kp, k)), np.concatenate((vp, v)), np.concatenate((okp, ok))
        limits = [prefix + n - T + t + 1 for t in range(T)]
        want, mag = R.attention(q[b], k, v, ok, limits, scale)
        err = np.abs(out[b] - want)
        bound = 2.0**-8 * np.abs(want) + 2.0**-9 * mag + 2.0**-126
        assert np.isfinite(out[b]).all(), f"sequence {b}"
        worst = max(worst, float((err / bound).max()))
    assert worst <= 1.0, worst
    return worst


def call(q4, q, cache, table, lens, fmt, scale=None, prefix_pages=None, prefix=0, **kw):
    c, t = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qd = bf16(q).cuda()
    if prefix:
        return q4.q4_kv_attention_shared(qd, c, torch.from_numpy(np.ascontiguousarray(prefix_pages)).cuda(), prefix,
                                         t, n, fmt, scale, **kw)
    return q4.q4_kv_attention(qd, c, t, n, fmt, scale, **kw)


SHAPES = [  # batch lengths, tokens, q_heads, kv_heads, page
    ([1], 1, 1, 1, 16),
    ([15, 16, 17, 31, 32, 33], 1, 4, 2, 16),
    ([0, 1, 63, 64, 65, 700], 1, 8, 1, 32),
    ([1000, 3], 1, 16, 16, 64),
    ([129, 5, 0, 257], 2, 6, 2, 128),                       # lengths below the query tokens
    ([2, 77, 300], 5, 14, 2, 16),                           # groups of 7
    ([4100], 1, 32, 4, 1024),
    ([513, 40], 33, 8, 2, 64),                              # a chunk
    ([260, 200, 130], 130, 3, 1, 32),                       # more rows than a tile
    ([290], 200, 4, 4, 16),
    ([20000, 3], 1, 34, 2, 64),                             # 17 rows, many tiles
    ([6, 70], 9, 30, 2, 32),                                # 135 rows: a tile of 128 and one of 7
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,T,Hq,H,page", SHAPES)
def test_attention_matches_fp64(q4, fmt, D, lens, T, Hq, H, page):
    rng = np.random.default_rng([5, fmt, D, T, Hq, len(lens)])
    cache, table, _ = filled(rng, fmt, D, H, page, lens)
    q = bf16(1.5 * rng.standard_normal((len(lens), T, Hq, D))).float().numpy()
    q4.device_error_flags(clear=True)
    out = call(q4, q, cache, table, lens, fmt)
    assert q4.device_error_flags() == 0
    check(out, q, cache, table, lens, fmt, D**-0.5)
    for b, n in enumerate(lens):                            # rows that see nothing
        for t in range(max(0, T - n)):
            assert not bits(out[b, t]).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,T,Hq,H,page,prefix", [
    ([1], 1, 1, 1, 16, 1),
    ([0, 5, 40], 1, 8, 2, 16, 33),
    ([0, 1, 2, 60], 4, 6, 2, 32, 100),                      # lengths below the query tokens
    ([17] * 40, 1, 16, 4, 64, 400),                         # more rows than a tile
    ([3, 200, 90], 65, 4, 2, 16, 257),
    ([64, 1], 1, 14, 2, 128, 1500),
])
def test_shared_prefix_matches_fp64(q4, fmt, D, lens, T, Hq, H, page, prefix):
    rng = np.random.default_rng([6, fmt, D, T, Hq, len(lens)])
    cache, table, pp = filled(rng, fmt, D, H, page, lens, prefix=prefix)
    q = bf16(1.5 * rng.standard_normal((len(lens), T, Hq, D))).float().numpy()
    q4.device_error_flags(clear=True)
    out = call(q4, q, cache, table, lens, fmt, None, pp, prefix)
    assert q4.device_error_flags() == 0
    check(out, q, cache, table, lens, fmt, D**-0.5, pp, prefix)


@pytest.mark.parametrize("fmt", FMTS)
def test_ranges_of_scales_and_queries(q4, fmt):
    """V scales and queries far from 1, tokens of very different V scale, one token that
    outweighs all others, and equal scores throughout."""
    rng = np.random.default_rng([7, fmt])
    D, H, page, lens = 128, 2, 32, [300, 300, 300, 300]
    cache, table, _ = filled(rng, fmt, D, H, page, lens)

    def put(b, k, v):
        pos = np.arange(300)
        R.write(cache, table[b][pos // page].astype(np.int64) * page + pos % page, k, v, fmt, page)

    k, v = rows(rng, 300, H, D), rows(rng, 300, H, D)
    put(0, k * np.float32(2**-6), v * np.float32(2.0**-10))
    put(1, k * np.float32(2**10), v * np.float32(2.0**18))
    put(2, np.broadcast_to(k[:1], k.shape), v * np.exp2(rng.integers(-8, 9, (300, 1, 1))).astype(np.float32))
    big = k.copy()
    big[123] *= 8
    put(3, big, v)
    q = bf16(rng.standard_normal((4, 1, 4, D))).float().numpy()
    q[0] *= 2**7
    q[1] *= 2.0**-11
    q[3, 0, :2] = big[123, 0] / 4
    q = bf16(q).float().numpy()
    out = call(q4, q, cache, table, lens, fmt)
    check(out, q, cache, table, lens, fmt, D**-0.5)


def test_poisoned_rows_reach_only_their_readers(q4):
    """A NaN row gives NaN to the rows that see it, and to no others."""
    rng = np.random.default_rng(8)
    D, H, page, lens = 64, 2, 16, [50, 60]
    cache, table, _ = filled(rng, 0, D, H, page, lens)
    bad = rows(rng, 1, H, D)
    bad[0, 1, 0] = np.nan
    R.write(cache, [int(table[0, 3]) * page + 1], rows(rng, 1, H, D), bad, 0, page)     # V of token 49, head 1
    q = rows(rng, 2 * 3, 4, D).reshape(2, 3, 4, D)
    out = call(q4, q, cache, table, lens, 0).float().cpu().numpy()
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[0, 2, 2:] = True                                   # the last query token, heads 2 and 3
    np.testing.assert_array_equal(nan, want)


@pytest.mark.parametrize("prefix", [0, 70])
def test_bad_pages_and_lengths_past_the_table(q4, prefix):
    rng = np.random.default_rng(9)
    D, H, page, lens = 128, 2, 16, [100, 64, 30]
    cache, table, pp = filled(rng, 0, D, H, page, lens, prefix=prefix)
    table[0, 2] = -5
    table[0, 4] = cache.shape[0]
    if prefix:
        pp = pp.copy()
        pp[1] = 10**6
    seen = [100, 64, 10**9]                                 # the table holds 112 tokens of each
    table[2] = table[0]
    q = rows(rng, 3, 4, D).reshape(3, 1, 4, D)
    q4.device_error_flags(clear=True)
    out = call(q4, q, cache, table, seen, 0, None, pp, prefix)
    assert q4.device_error_flags() == 4
    check(out[:2], q[:2], cache, table[:2], seen[:2], 0, D**-0.5, pp, prefix)
    assert np.isfinite(out.float().cpu().numpy()[:2]).all()


@pytest.mark.parametrize("shared", [False, True])
def test_repeated_captured_and_streamed_calls_agree(q4, shared):
    """The same bits again on a used workspace, on another stream, from a replayed graph
    whose lengths grow, and with programmatic dependent launch."""
    rng = np.random.default_rng(10)
    D, H, page, lens, prefix = 128, 4, 16, [900, 33, 1, 400], 300 if shared else 0
    cache, table, pp = filled(rng, 1, D, H, page, lens, prefix=prefix)
    q = rows(rng, 4 * 2, 8, D).reshape(4, 2, 8, D)
    first = bits(call(q4, q, cache, table, lens, 1, None, pp, prefix))
    np.testing.assert_array_equal(bits(call(q4, q, cache, table, lens, 1, None, pp, prefix)), first)
    c, t, qd = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), bf16(q).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ppd = torch.from_numpy(np.ascontiguousarray(pp)).cuda()

    def go(**kw):
        return q4.q4_kv_attention_shared(qd, c, ppd, prefix, t, n, 1, **kw) if shared else \
            q4.q4_kv_attention(qd, c, t, n, 1, **kw)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = go(stream=side)
    side.synchronize()
    np.testing.assert_array_equal(bits(out), first)
    try:
        q4.set_launch_flags(q4.FLAG_PDL)
        out = [go() for _ in range(3)][-1]
        np.testing.assert_array_equal(bits(out), first)
        with torch.cuda.stream(side):
            go()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            out = torch.empty_like(qd)
            with torch.cuda.graph(graph, stream=side):
                go(out=out)
                go(out=out)
        for step in range(3):
            n.copy_(torch.tensor([900 - step, 33, 1 + step, 400 - 3 * step], dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            got = bits(out)
            np.testing.assert_array_equal(got, bits(go()))
            if step == 0:
                np.testing.assert_array_equal(got, first)
    finally:
        q4.set_launch_flags(0)


@pytest.mark.parametrize("Hq", [4, 40])
def test_a_call_captured_before_any_has_run(q4, Hq):
    """The workspace that such a call gets is filled in its graph; calls between capture and
    replay have one of their own."""
    rng = np.random.default_rng([16, Hq])
    lens = [611, 1999, 5]
    cache, table, _ = filled(rng, 1, 128, 2, 32, lens)
    q = bf16(rng.standard_normal((3, 1, Hq, 128))).cuda()
    c, t = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = q4.q4_kv_attention(q, c, t, n, 1)
    with torch.cuda.stream(stream):
        between = bits(q4.q4_kv_attention(q, c, t, n, 1))
        for _ in range(2):
            graph.replay()
            np.testing.assert_array_equal(bits(captured), between)
        np.testing.assert_array_equal(bits(q4.q4_kv_attention(q, c, t, n, 1)), between)
    check(captured, q.float().cpu().numpy(), cache, table, lens, 1, 128**-0.5)


@pytest.mark.parametrize("Hq", [4, 40])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-9])
def test_scales_of_any_sign(q4, scale, Hq):
    rng = np.random.default_rng([13, Hq])
    cache, table, _ = filled(rng, 0, 64, 2, 16, [200, 131])
    q = rows(rng, 2, Hq, 64).reshape(2, 1, Hq, 64)
    out = call(q4, q, cache, table, [200, 131], 0, scale)
    check(out, q, cache, table, [200, 131], 0, float(np.float32(scale)))


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("fmt", FMTS)
def test_query_rows_of_very_different_size(q4, fmt, T):
    """Rows of one key head whose sizes lie 2^48 apart: no row takes another one's digits."""
    rng = np.random.default_rng([14, fmt, T])
    lens = [300, 140]
    cache, table, _ = filled(rng, fmt, 64, 2, 16, lens)
    q = bf16(1.5 * rng.standard_normal((2, T, 4, 64))).float().numpy()
    q[:, :, 1] *= np.float32(2.0**-48)
    out = call(q4, q, cache, table, lens, fmt)
    check(out, q, cache, table, lens, fmt, 0.125)
    q[:, :, 0] *= np.float32(2.0**48)                       # (one token takes all: any rounding may pick another)
    out = call(q4, q, cache, table, lens, fmt)[:, :, 1:2]
    # head 1 alone, as the head of a cache that has only its key head
    check(out, q[:, :, 1:2], np.ascontiguousarray(cache[:, :1]), table, lens, fmt, 0.125)


def test_query_rows_of_a_fused_projection(q4):
    rng = np.random.default_rng(11)
    D, H, Hq, page, lens = 64, 2, 6, 32, [70, 20]
    cache, table, _ = filled(rng, 0, D, H, page, lens)
    wide = bf16(rng.standard_normal((2 * 3, (Hq + 2 * H) * D))).cuda()
    q = wide[:, H * D:(H + Hq) * D].view(2, 3, Hq, D)
    out = q4.q4_kv_attention(q, torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), 0, 0.3)
    check(out, q.float().cpu().numpy(), cache, table, lens, 0, np.float64(np.float32(0.3)))


def test_cache_of_more_than_4_gib(q4):
    """Pages whose first byte lies past 2^32 are written, read and attended to."""
    rng = np.random.default_rng(12)
    D, H, page, n = 128, 16, 1024, 40
    pages = (1 << 32) // (H * page // 16 * R.block_bytes(0, D)) + 3
    cache = q4.alloc_kv_cache(0, pages, page, H, D)
    assert cache.numel() > 1 << 32
    k, v = rows(rng, n, H, D), rows(rng, n, H, D)
    last = pages - 1
    slots = torch.arange(n, dtype=torch.int32, device="cuda") + last * page
    q4.q4_kv_write(bf16(k).cuda(), bf16(v).cuda(), cache, slots, 0)
    table = torch.tensor([[last]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    small = np.zeros((1, H, page // 16, R.block_bytes(0, D)), np.uint8)
    R.write(small, np.arange(n), k, v, 0, page)
    np.testing.assert_array_equal(cache[last, :, :n // 16].cpu().numpy(), small[0, :, :n // 16])
    kk, vv, _ = R.read(small, [0], n, 0, D)
    got = q4.q4_kv_read(cache, table, lens, n, D, 0)
    same_bf16(got[0][0], kk)
    same_bf16(got[1][0], vv)
    q = rows(rng, 1, H, D).reshape(1, 1, H, D)
    out = q4.q4_kv_attention(bf16(q).cuda(), cache, table, lens, 0)
    check(out, q, small, np.zeros((1, 1), np.int32), [n], 0, D**-0.5)


def test_binding_refuses_what_the_kernels_do_not_take(q4):
    c = q4.alloc_kv_cache(0, 4, 16, 2, 64)
    t = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [lambda: q4.q4_kv_attention(q.float(), c, t, n, 0), lambda: q4.q4_kv_attention(q, c, t, n, 1),
           lambda: q4.q4_kv_attention(q, c, t.long(), n, 0), lambda: q4.q4_kv_attention(q, c, t[0], n, 0),
           lambda: q4.q4_kv_attention(q.transpose(2, 3), c, t, n, 0),
           lambda: q4.q4_kv_attention(q.expand(2, 1, 4, 64), c, t, n, 0),
           lambda: q4.q4_kv_attention(q, c, t, n, 0, out=q[:, :, :2]),
           lambda: q4.q4_kv_attention_shared(q, c, t[0], 33, t, n, 0),
           lambda: q4.q4_kv_attention_shared(q, c, t[0], 0, t, n, 0),
           lambda: q4.q4_kv_write(k, k[:, :, :32], c, s, 0), lambda: q4.q4_kv_write(k, k, c, s[:2], 0),
           lambda: q4.q4_kv_write(k[:, :1], k[:, :1], c, s, 0), lambda: q4.q4_kv_write(k, k, c, s.long(), 0),
           lambda: q4.q4_kv_read(c, t, n, 4, 128, 0), lambda: q4.q4_kv_read(c, t, n[:0], 4, 64, 0),
           lambda: q4.q4_kv_read(c, t, n, 4, 64, 0, k=k), lambda: q4.alloc_kv_cache(0, 4, 24, 2, 64),
           lambda: q4.alloc_kv_cache(0, 4, 16, 2, 96), lambda: q4.alloc_kv_cache(2, 4, 16, 2, 64)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(q4.Q4Error):
        q4.q4_kv_attention(q[:, :, :3], c, t, n, 0)         # 3 query heads on 2
    with pytest.raises(q4.Q4Error):
        q4.q4_kv_attention(q, c, t, n, 0, scale=float("inf"))
