"""Refusals of the operators around a layer's projections that come before any launch (fake pointers are
never dereferenced, and no device is asked for): 1 NULL, 2 shape, 3 alignment, 5 argument."""
import ctypes

import pytest
import torch

from bit_weight_only_q4_gb300 import build as q4build
from bit_weight_only_q4_gb300 import q4

FAKE = 1 << 20
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load()


def rope(lib, q=FAKE, qs=512, qw=FAKE, qo=FAKE, qos=512, Hq=8, k=FAKE, ks=128, kw=FAKE, ko=FAKE, kos=128, H=2, pos=FAKE,
         freq=FAKE, rotary=64, inter=0, eps=1e-6, tokens=3, D=64):
    return lib.q4_norm_rope(q, qs, qw, qo, qos, Hq, k, ks, kw, ko, kos, H, pos, freq, rotary, inter, ctypes.c_float(eps),
                            tokens, D, None)


def test_norm_rope(lib):
    assert rope(lib, q=None) == 1 and rope(lib, ko=None) == 1 and rope(lib, pos=None) == 1 and rope(lib, freq=None) == 1
    assert rope(lib, D=96) == 2 and rope(lib, tokens=0) == 2 and rope(lib, Hq=-1) == 2 and rope(lib, H=70000) == 2
    assert rope(lib, Hq=0, H=0) == 2
    for rotary in (-16, 8, 40, 80):
        assert rope(lib, rotary=rotary) == 2
    for name in ("qs", "qos", "ks", "kos"):
        assert rope(lib, **{name: 120}) == 2 and rope(lib, **{name: 516}) == 2 and rope(lib, **{name: -512}) == 2
    for name in ("q", "k", "qo", "ko", "qw", "kw"):
        assert rope(lib, **{name: FAKE + 8}) == 3
    assert rope(lib, pos=FAKE + 2) == 3 and rope(lib, freq=FAKE + 1) == 3
    assert rope(lib, inter=2) == 5
    for eps in (-1e-9, INF, float("nan")):
        assert rope(lib, eps=eps) == 5
    assert rope(lib, qos=520) == 5                           # in place, but other strides
    assert b"in place" in lib.q4_last_error_string()


def prompt(lib, q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, offsets=FAKE, batch=2, tokens=10, Hq=8, H=2, D=64, scale=0.1,
           out=FAKE):
    return lib.q4_prompt_attention(q, qs, k, ks, v, vs, offsets, batch, tokens, Hq, H, D, ctypes.c_float(scale), out, None)


def test_prompt_attention(lib):
    for name in ("q", "k", "v", "offsets", "out"):
        assert prompt(lib, **{name: None}) == 1
    for change in (dict(D=32), dict(batch=0), dict(tokens=0), dict(Hq=0), dict(H=0), dict(Hq=7), dict(Hq=1), dict(qs=504),
                   dict(ks=124), dict(vs=132), dict(qs=1 << 40), dict(tokens=(1 << 31) - 1),
                   dict(batch=1 << 30), dict(Hq=258, qs=258 * 64), dict(ks=-128)):
        assert prompt(lib, **change) == 2, change
    for name in ("q", "k", "v", "out"):
        assert prompt(lib, **{name: FAKE + 8}) == 3
    assert prompt(lib, offsets=FAKE + 2) == 3
    for scale in (INF, -INF, float("nan")):
        assert prompt(lib, scale=scale) == 5


def lora(lib, x=FAKE, xs=64, a=FAKE, b=FAKE, scales=FAKE, n=2, rank=16, offsets=FAKE, ids=FAKE, batch=3, base=FAKE, bs=128,
         out=FAKE + 4096, outs=128, M=10, N=128, K=64):
    return lib.q4_lora(x, xs, a, b, scales, n, rank, offsets, ids, batch, base, bs, out, outs, M, N, K, None)


def test_lora(lib):
    for name in ("x", "a", "b", "scales", "offsets", "ids", "base", "out"):
        assert lora(lib, **{name: None}) == 1
    for change in (dict(n=0), dict(batch=0), dict(M=0), dict(N=0), dict(K=0), dict(N=124), dict(K=60), dict(rank=0), dict(rank=4),
                   dict(rank=20), dict(rank=136), dict(rank=-8), dict(xs=56), dict(xs=68), dict(bs=120), dict(outs=120),
                   dict(outs=132), dict(M=1 << 27), dict(batch=1 << 27), dict(bs=1 << 40)):
        assert lora(lib, **change) == 2, change
    for name in ("x", "a", "b", "base", "out"):
        assert lora(lib, **{name: FAKE + 8}) == 3
    for name in ("scales", "offsets", "ids"):
        assert lora(lib, **{name: FAKE + 2}) == 3
    assert lora(lib, out=FAKE, outs=136) == 5


def test_results_over_other_inputs(lib):
    assert rope(lib, k=2 * FAKE, ko=2 * FAKE, q=FAKE, qo=2 * FAKE) == 5
    assert rope(lib, k=2 * FAKE, ko=FAKE, q=FAKE, qo=3 * FAKE) == 5
    assert rope(lib, k=2 * FAKE, ko=3 * FAKE, q=FAKE, qo=3 * FAKE) == 5
    for name in ("q", "k", "v"):
        assert prompt(lib, **dict(dict(q=2 * FAKE, k=2 * FAKE, v=2 * FAKE), **{name: FAKE})) == 5
    for name in ("x", "a", "b"):
        assert lora(lib, **{name: FAKE + 4096}) == 5


def test_host_tensors_are_refused():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)      # noqa: E731
    with pytest.raises(ValueError):
        q4.q4_norm_rope(bf(3, 2, 64), bf(3, 1, 64), None, None, None, None)
    with pytest.raises(ValueError):
        q4.q4_prompt_attention(bf(3, 2, 64), bf(3, 1, 64), bf(3, 1, 64), i32(2))
    with pytest.raises(ValueError):
        q4.q4_lora(bf(3, 64), bf(1, 8, 64), bf(1, 32, 8), torch.zeros(1), i32(2), i32(1), bf(3, 32))
