"""The key/value cache and its attention at the edges: inputs, shapes and ways of calling that
test_gpu_kv_cache.py does not reach.  Its helpers and its bound (see there) are used throughout."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import kv_reference as R
from tests.test_gpu_kv_cache import FMTS, bf16, bits, call, filled, q4, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,H", [(1, 40, 2), (9, 4, 2), (43, 6, 2)])
def test_many_short_units_of_many_rows(q4, fmt, D, T, Hq, H):
    """Units of one tile whose row tile is filled by 20, 18 and 129 rows (warps without rows beside
    warps with), several to a CTA: the same bits every time, and those of each sequence by itself."""
    rng = np.random.default_rng([20, fmt, D, T])
    lens = [int(n) for n in rng.integers(1, 129, 400)]
    cache, table, _ = filled(rng, fmt, D, H, 16, lens)
    q = bf16(1.5 * rng.standard_normal((len(lens), T, Hq, D))).float().numpy()
    out = call(q4, q, cache, table, lens, fmt)
    first = bits(out)
    for _ in range(4):
        np.testing.assert_array_equal(bits(call(q4, q, cache, table, lens, fmt)), first)
    # a sequence's units are whole here, so alone it takes the same steps in the same order
    for b in range(0, len(lens), 25):
        np.testing.assert_array_equal(bits(call(q4, q[b:b + 1], cache, table[b:b + 1], lens[b:b + 1], fmt)), first[b:b + 1])


GIVE_UP = [  # tokens, q_heads, prefix: the few-row kernel, the many-row kernel, one after the other
    (1, 8, 0), (5, 16, 0), (1, 8, 300)]


def some_calls(q4, fmt, T, Hq, prefix):
    """A batch of split and whole units and a way to attend to it: go(**kw)."""
    rng = np.random.default_rng([21, fmt, T, Hq])
    D, H, page, lens = 128, 2, 32, [700, 12000, 60, 9000]
    cache, table, pp = filled(rng, fmt, D, H, page, lens, prefix=prefix)
    c, t, p = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(pp).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = bf16(rng.standard_normal((len(lens), T, Hq, D))).cuda()
    size = q4.kv_attention_workspace_bytes(fmt, H, D, len(lens), T, Hq, prefix)

    def go(**kw):
        return q4.q4_kv_attention_shared(q, c, p, prefix, t, n, fmt, **kw) if prefix else \
            q4.q4_kv_attention(q, c, t, n, fmt, **kw)
    return go, size


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,Hq,prefix", GIVE_UP)
@pytest.mark.parametrize("cta,tiles", [(0, 0), (0, 1), (3, 0), (1, 3)])
def test_a_cta_that_gives_up_ends_the_call_with_a_status(q4, fmt, T, Hq, prefix, cta, tiles):
    """Before its first unit has been described, or in the midst of one."""
    go, size = some_calls(q4, fmt, T, Hq, prefix)
    q4.device_error_flags(clear=True)
    try:
        q4.load().q4_test_kv_give_up(cta, tiles)
        go(workspace=torch.zeros(size, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
    finally:
        q4.load().q4_test_kv_give_up(-1, 0)
    assert q4.device_error_flags() == 1
    go(workspace=torch.zeros(size, dtype=torch.uint8, device="cuda"))
    assert q4.device_error_flags() == 0


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("fmt", FMTS)
def test_one_workspace_serves_calls_of_every_shape(q4, fmt, prefix):
    """A buffer of the largest size, zero-filled once: few sequences, many, more rows, few again."""
    rng = np.random.default_rng([22, fmt])
    D, H, page = 128, 16, 64
    mixed = [100 + 97 * b % 1500 for b in range(160)]
    shapes = [([2047], 1, 16), (mixed, 1, 16), (mixed, 2, 32), ([900, 2047], 5, 64), ([2047], 1, 16)]
    cache, table, pp = filled(rng, fmt, D, H, page, [2047] * 2, prefix=prefix)
    c, p = torch.from_numpy(cache).cuda(), torch.from_numpy(pp).cuda()

    def go(lens, T, Hq, ws):
        t = torch.from_numpy(np.ascontiguousarray(table[np.arange(len(lens)) % 2])).cuda()
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = bf16(np.random.default_rng(Hq).standard_normal((len(lens), T, Hq, D))).cuda()
        out = torch.full_like(q, torch.nan)
        if prefix:
            q4.q4_kv_attention_shared(q, c, p, prefix, t, n, fmt, out=out, workspace=ws)
        else:
            q4.q4_kv_attention(q, c, t, n, fmt, out=out, workspace=ws)
        return bits(out)

    size = [q4.kv_attention_workspace_bytes(fmt, H, D, len(n), T, Hq, prefix) for n, T, Hq in shapes]
    one = torch.zeros(max(size), dtype=torch.uint8, device="cuda")
    for (lens, T, Hq), n in zip(shapes, size):
        want = go(lens, T, Hq, torch.zeros(n, dtype=torch.uint8, device="cuda"))
        np.testing.assert_array_equal(go(lens, T, Hq, one), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,Hq,prefix", GIVE_UP)
def test_a_workspace_stays_usable_after_a_cta_gave_up(q4, fmt, T, Hq, prefix):
    go, size = some_calls(q4, fmt, T, Hq, prefix)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = bits(go(workspace=ws))
    for cta, tiles in ((0, 0), (2, 1), (60, 2), (7, 3)):
        try:
            q4.load().q4_test_kv_give_up(cta, tiles)
            go(workspace=ws)
            torch.cuda.synchronize()
        finally:
            q4.load().q4_test_kv_give_up(-1, 0)
        assert q4.device_error_flags() == 1
        assert not ws[:4096].any()
        out = torch.full(want.shape, torch.nan, dtype=torch.bfloat16, device="cuda")
        np.testing.assert_array_equal(bits(go(out=out, workspace=ws)), want)
        assert q4.device_error_flags() == 0


@pytest.mark.parametrize("T", [1, 9])
def test_host_threads_on_one_stream_and_workspace(q4, T):
    """Calls with a shared prefix (two launches) from several threads on the default stream, beside
    calls without one: each gets its own results."""
    import threading
    rng = np.random.default_rng([23, T])
    D, H, Hq, page, lens, prefix, fmt = 64, 2, 8, 16, [40, 3, 200], 500, 1
    cache, table, pp = filled(rng, fmt, D, H, page, lens, prefix=prefix)
    c, t, p = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(pp).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    size = q4.kv_attention_workspace_bytes(fmt, H, D, len(lens), T, Hq, prefix)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    qs = [bf16(rng.standard_normal((len(lens), T, Hq, D))).cuda() for _ in range(4)]

    def go(i):
        if i == 3:
            return q4.q4_kv_attention(qs[i], c, t, n, fmt, workspace=ws)
        return q4.q4_kv_attention_shared(qs[i], c, p, prefix, t, n, fmt, workspace=ws)

    want = [bits(go(i)) for i in range(4)]
    out = [[] for _ in range(4)]
    threads = [threading.Thread(target=lambda i=i: out[i].extend(go(i) for _ in range(300))) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    for got, w in zip(out, want):
        assert len(got) == 300
        for o in got:
            np.testing.assert_array_equal(bits(o), w)


@pytest.mark.parametrize("prefix", [0, 130])
@pytest.mark.parametrize("explicit", [False, True])
def test_a_graph_keeps_its_workspace(q4, prefix, explicit):
    """A call captured after an eager one, then a hundred calls of other shapes and memory that is taken and
    filled: the replay gives the same bits and touches nothing of that memory."""
    rng = np.random.default_rng([24, prefix])
    D, H, Hq, page, lens, fmt = 128, 2, 8, 32, [9000, 700], 1
    cache, table, pp = filled(rng, fmt, D, H, page, lens, prefix=prefix)
    c, t, p = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(pp).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = bf16(rng.standard_normal((2, 1, Hq, D))).cuda()
    big = bf16(rng.standard_normal((2, 100, 4 * Hq, D))).cuda()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    kw = dict(stream=side) if explicit else {}

    def go(q, prefix, **kw):
        return q4.q4_kv_attention_shared(q, c, p, prefix, t, n, fmt, **kw) if prefix else \
            q4.q4_kv_attention(q, c, t, n, fmt, **kw)

    with torch.cuda.stream(side):
        want = bits(go(q, prefix, **kw))
        with torch.cuda.graph(graph, stream=side):
            out = go(q, prefix, **kw)
            assert q4._capture_id(side.cuda_stream, kw.get("stream")) != 0
        assert q4._capture_id(side.cuda_stream, kw.get("stream")) == 0
        for T in range(1, 101):                             # more rows, and more room, from call to call
            go(big[:, :T].contiguous(), max(0, prefix - T), **kw)
        side.synchronize()
        torch.cuda.empty_cache()
        taken = [torch.full((m << 20,), 0x5a, dtype=torch.uint8, device="cuda") for m in (1, 2, 4, 8, 16, 20, 24, 40) * 3]
        for _ in range(2):
            graph.replay()
            np.testing.assert_array_equal(bits(out), want)
        assert all(bool((x == 0x5a).all()) for x in taken)
        np.testing.assert_array_equal(bits(go(q, prefix, **kw)), want)


def test_calls_of_one_cold_capture(q4):
    """Several shapes captured before any call has run on the stream, beside eager calls of theirs."""
    rng = np.random.default_rng(25)
    D, H, page, lens, fmt = 64, 2, 16, [3000, 90], 0
    cache, table, _ = filled(rng, fmt, D, H, page, lens)
    c, t = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [bf16(rng.standard_normal((2, T, 8, D))).cuda() for T in (1, 20, 2, 60, 1)]
    want = [bits(q4.q4_kv_attention(q, c, t, n, fmt)) for q in qs]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = [q4.q4_kv_attention(q, c, t, n, fmt) for q in qs]
    with torch.cuda.stream(side):
        for _ in range(3):
            for q, w in zip(qs, want):
                np.testing.assert_array_equal(bits(q4.q4_kv_attention(q, c, t, n, fmt)), w)
            graph.replay()
            for o, w in zip(outs, want):
                np.testing.assert_array_equal(bits(o), w)


def past_the_table(q, cache, table, lens, fmt, scale, prefix_pages=(), prefix=0):
    """The definition where a length goes past the table: query token t sees the positions below
    prefix + lengths[b] - tokens + t + 1 of those that the table holds."""
    B, T, Hq, D = q.shape
    cap = table.shape[1] * cache.shape[2] * 16
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        k, v, ok = R.read(cache, table[b], n, fmt, D)
        if prefix:
            kp, vp, okp = R.read(cache, prefix_pages, prefix, fmt, D)
            k, v, ok = np.concatenate((kp, k)), np.concatenate((vp, v)), np.concatenate((okp, ok))
        limits = [prefix + max(int(lens[b]), 0) - T + t + 1 for t in range(T)]
        out[b], mag[b] = R.attention(q[b], k, v, ok, limits, scale)
    return out, mag


@pytest.mark.parametrize("T,Hq", [(3, 4), (20, 2), (20, 20)])
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("D", [64, 128])
def test_query_tokens_of_lengths_past_the_table(q4, D, prefix, T, Hq):
    """The table holds 48 tokens of each sequence: all of them are seen where the length lets the
    query token see them, and the token's own place may lie past the table."""
    rng = np.random.default_rng([26, D, T, Hq])
    fmt, H, page = 0, 2, 16
    cache, table, pp = filled(rng, fmt, D, H, page, [48] * 7, prefix=prefix)
    lens = [100, 48, 49, 48 + T, 48 + T - 1, 2**31 - 1, -5]
    q = bf16(1.5 * rng.standard_normal((7, T, Hq, D))).float().numpy()
    q4.device_error_flags(clear=True)
    out = call(q4, q, cache, table, lens, fmt, None, pp, prefix)
    assert q4.device_error_flags() == 4
    got = out.float().cpu().numpy().astype(np.float64)
    want, mag = past_the_table(q, cache, table, lens, fmt, D**-0.5, pp, prefix)
    assert (np.abs(got - want) <= 2.0**-8 * np.abs(want) + 2.0**-9 * mag + 2.0**-126).all()


def within(out, q, caches, table, lens, fmt, scale):
    """The bound of test_gpu_kv_cache.py, in units of which the worst element is off."""
    got = out.float().cpu().numpy().astype(np.float64)
    want, mag = past_the_table(q, caches, table, lens, fmt, scale)
    return float((np.abs(got - want) / (2.0**-8 * np.abs(want) + 2.0**-9 * mag + 2.0**-126)).max())


def put(cache, pages, page, at, k, v, fmt):
    """Rows k, v [n, H, D] as tokens at, at + 1, ... of a list of pages."""
    pos = at + np.arange(len(k))
    R.write(cache, pages[pos // page].astype(np.int64) * page + pos % page, k, v, fmt, page)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq", [(4, 4), (40, 4)])
@pytest.mark.parametrize("power", [14, 22, 30])
def test_later_tokens_take_no_digits_from_earlier_rows(q4, fmt, D, T, Hq, power):
    """A chunk whose last token's V is 2^power times the others': the rows that do not see it give
    the bits that they give without it."""
    rng = np.random.default_rng([27, fmt, D, T])
    H, page, n = 2, 16, 100
    cache, table, _ = filled(rng, fmt, D, H, page, [n])
    k, v = rows(rng, n, H, D), rows(rng, n, H, D) * np.float32(2.0**-14)
    put(cache, table[0], page, 0, k, v, fmt)
    q = bf16(1.5 * rng.standard_normal((1, T, Hq, D))).float().numpy()
    want = bits(call(q4, q, cache, table, [n], fmt))[:, :-1]
    put(cache, table[0], page, n - 1, k[-1:], v[-1:] * np.float32(2.0**power), fmt)
    np.testing.assert_array_equal(bits(call(q4, q, cache, table, [n], fmt))[:, :-1], want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq", [(1, 4), (1, 40), (9, 4)])
@pytest.mark.parametrize("small,weight,up", [(-6, 24, 0), (-14, 24, 0), (-20, 24, 0), (-24, 40, 8), (-28, 44, 10)])
def test_the_token_that_counts_may_have_the_smallest_values(q4, D, T, Hq, small, weight, up):
    """One token outweighs all others by far and has a V 2^small times theirs
    (which are of the size 2^up)."""
    rng = np.random.default_rng([28, D, T, Hq])
    fmt, H, page, n = 0, 2, 32, 400
    cache, table, _ = filled(rng, fmt, D, H, page, [n])
    k, v = 0.1 * rows(rng, n, H, D), rows(rng, n, H, D) * np.float32(2.0**up)
    k[77] = 1.0
    v[77] *= np.float32(2.0**small)
    put(cache, table[0], page, 0, k, v, fmt)
    q = bf16(0.1 * rng.standard_normal((1, T, Hq, D)) + 1.0).float().numpy()
    scale = weight * np.log(2.0) / D                        # 2^weight times the others' weight
    out = call(q4, q, cache, table, [n], fmt, scale)
    assert within(out, q, cache, table, [n], fmt, float(np.float32(scale))) <= 1.0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq", [(1, 4), (1, 40), (9, 4)])
@pytest.mark.parametrize("rise,value", [(20, 1.0), (60, -300.0), (84, 1.0), (87, 300.0), (90, -1.0), (91, 300.0), (130, 1.0)])
def test_constant_values_under_rising_scores(q4, fmt, D, T, Hq, rise, value):
    """V rows that are one value throughout (int4: scale 0, the minimum says it all), and scores that rise
    by 2^rise from the first tiles to later ones: the result is that value.  A hundred sequences on
    the same pages, so that a CTA meets the rise within a unit."""
    rng = np.random.default_rng([29, fmt, D, T])
    H, page, n, B = 2, 32, 1000, 100
    cache, table, _ = filled(rng, fmt, D, H, page, [n])
    k, v = 0.01 * rows(rng, n, H, D), np.full((n, H, D), value, np.float32)
    k[500:] += 1.0
    put(cache, table[0], page, 0, k, v, fmt)
    table = np.repeat(table, B, 0)
    q = bf16(0.01 * rng.standard_normal((B, T, Hq, D)) + 1.0).float().numpy()
    scale = rise * np.log(2.0) / D
    out = call(q4, q, cache, table, [n] * B, fmt, scale)
    got = out.float().cpu().numpy()
    # (weights that add up to one: the bound is 2^-8 |value| + 2^-9 |value|)
    assert np.isfinite(got).all() and (np.abs(got - value) <= 1.5 * 2.0**-8 * abs(value)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq", [(1, 4), (1, 40)])
@pytest.mark.parametrize("weight", [30, 60, 72])
def test_values_of_zero_beside_others(q4, D, T, Hq, weight):
    """Tokens whose V is zero outweigh the others by 2^weight: what is left is the others' share."""
    rng = np.random.default_rng([30, D, T])
    fmt, H, page, n, B = 0, 2, 32, 1000, 40
    cache, table, _ = filled(rng, fmt, D, H, page, [n])
    k, v = np.zeros((n, H, D), np.float32), rows(rng, n, H, D)
    k[500:] = 1.0
    v[500:] = 0.0
    put(cache, table[0], page, 0, k, v, fmt)
    table = np.repeat(table, B, 0)
    q = np.ones((B, T, Hq, D), np.float32)
    scale = weight * np.log(2.0) / D
    out = call(q4, q, cache, table, [n] * B, fmt, scale)
    some = slice(0, B, 8)
    assert within(out[some], q[some], cache, table[some], [n] * len(q[some]), fmt, float(np.float32(scale))) <= 1.0


def test_layer_with_rotary_positions(q4):
    """project(), a turn of q and k by their positions, attend(): a prompt of two chunks and a single
    token give what one chunk of all gives, and what plain attention over the turned rows gives."""
    from bit_weight_only_q4_gb300 import cached_attention as C
    gen = torch.Generator("cuda").manual_seed(5)
    H, Hq, D, page, n = 2, 4, 64, 16, 45
    weights = C._weights((Hq + 2 * H) * D, 256, gen), C._weights(256, Hq * D, gen)
    x = torch.randn(1, n, 256, device="cuda", generator=gen).bfloat16()
    table = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")

    def turn(t, pos):                                       # [..., tokens, heads, D]
        angle = pos.view(-1, 1, 1) * 10.0 ** (-torch.arange(D // 2, device="cuda") / 8)
        a, b = t.float().chunk(2, -1)
        return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1).bfloat16()

    seen = []

    def run(cuts):
        layer = C.CachedAttention(*weights, Hq, q4.alloc_kv_cache(0, 3, page, H, D), 0, D)
        out = []
        for a, b in zip(cuts, cuts[1:]):
            pos = torch.arange(a, b, device="cuda").float()
            q, k, v = layer.project(x[:, a:b].contiguous())
            q, k = turn(q, pos), turn(k, pos)
            if cuts[1] == n:
                seen.extend((q, k, v))
            out.append(layer.attend(q, k, v, slots[a:b], table, torch.tensor([b], dtype=torch.int32, device="cuda")))
        return layer, torch.cat(out, 1)

    layer, whole = run((0, n))
    _, parts = run((0, 20, n - 1, n))
    # two roundings of the attention's output to bf16 apart, through one projection of 256 columns
    assert (parts.float() - whole.float()).abs().max() <= 2.0**-6 * whole.float().abs().max()
    q = seen[0].float().cpu().numpy()
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = q4.q4_kv_attention(seen[0], layer.cache, table, length, 0)
    assert within(got, q, layer.cache.cpu().numpy(), table.cpu().numpy(), [n], 0, D**-0.5) <= 1.0
