"""Host-side checks of the key/value cache entry points: sizes, and refusals before any
launch (fake pointers are never dereferenced)."""
import ctypes

import numpy as np
import pytest

from bit_weight_only_q4_gb300 import build as q4build
from bit_weight_only_q4_gb300 import q4
from tests import kv_reference as R

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load()


def test_block_bytes(lib):
    for fmt in (0, 1):
        for D in (64, 128):
            assert lib.q4_kv_block_bytes(fmt, D) == R.block_bytes(fmt, D) == q4.kv_block_bytes(fmt, D)
    assert lib.q4_kv_block_bytes(2, 64) == 0
    assert lib.q4_kv_block_bytes(0, 96) == 0
    assert lib.q4_kv_block_bytes(1, 0) == 0


def test_layout_is_a_permutation():
    for fmt in (0, 1):
        for D in (64, 128):
            rb = R.row_bytes(fmt, D)
            at = sorted(R.place(fmt, D, r, b) for r in range(16) for b in range(rb))
            assert at == list(range(16 * rb))


@pytest.mark.parametrize("fmt", [0, 1])
def test_reference_round_trip_error(fmt):
    """A value reads back within half a step of its row (and the fp16 rounding of scale and min)."""
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((50, 2, 64)).astype(np.float32)
    cache = np.zeros((4, 2, 1, R.block_bytes(fmt, 64)), np.uint8)
    R.write(cache, np.arange(50), x, -x, fmt, 16)
    k, v, ok = R.read(cache, np.arange(4), 50, fmt, 64)
    assert ok.all()
    span = np.abs(x).max(2, keepdims=True) / 127 if fmt == 0 else (x.max(2, keepdims=True) - x.min(2, keepdims=True)) / 15
    slack = 2.0**-11 * np.abs(x).max() * (2 if fmt else 1) + 1e-6
    assert (np.abs(k - x) <= 0.5 * span * (1 + 2.0**-10) + slack).all()
    assert (np.abs(v + x) <= 0.5 * span * (1 + 2.0**-10) + slack).all()


def _write(lib, k=FAKE, ks=512, v=FAKE, vs=512, slots=FAKE, n=3, cache=FAKE, fmt=0, pages=4, page=16,
           H=2, D=128):
    return lib.q4_kv_write(k, ks, v, vs, slots, n, cache, fmt, pages, page, H, D, None)


def _read(lib, cache=FAKE, fmt=0, pages=4, page=16, H=2, D=128, table=FAKE, width=2, lens=FAKE, B=1,
          most=20, k=FAKE, v=FAKE):
    return lib.q4_kv_read(cache, fmt, pages, page, H, D, table, width, lens, B, most, k, v, None)


def _attend(lib, q=FAKE, qs=512, cache=FAKE, fmt=0, pages=4, page=16, H=2, D=128, table=FAKE, width=2,
            lens=FAKE, B=1, T=1, Hq=4, scale=0.1, out=FAKE):
    return lib.q4_kv_attention(q, qs, cache, fmt, pages, page, H, D, table, width, lens, B, T, Hq,
                               ctypes.c_float(scale), out, None, 0, None)


def _shared(lib, pp=FAKE, prefix=20, width=2, **kw):
    return lib.q4_kv_attention_shared(FAKE, 512, FAKE, 0, 4, 16, 2, 128, pp, prefix, FAKE, width, FAKE, 1, 1, 4,
                                      ctypes.c_float(0.1), FAKE, None, 0, None)


@pytest.mark.parametrize("f", [_write, _read, _attend])
def test_invalid_caches_are_rejected(lib, f):
    assert f(lib, cache=None) == 1
    assert f(lib, fmt=2) == 5 and f(lib, fmt=-1) == 5
    assert f(lib, D=96) == 2 and f(lib, D=256) == 2
    assert f(lib, pages=0) == 2 and f(lib, H=0) == 2
    for page in (0, 8, 24, 48, 2048, -16):
        assert f(lib, page=page) == 2
    assert f(lib, cache=FAKE + 8) == 3


@pytest.mark.parametrize("f", [_write, _read, _attend])
def test_caches_of_too_many_blocks_are_rejected(lib, f):
    # (one more than 2^31 - 1 blocks of 16 tokens and a head)
    assert f(lib, pages=1 << 30, H=2) == 2
    assert f(lib, pages=1 << 24, H=2, page=1024) == 2
    assert b"blocks" in lib.q4_last_error_string()


def test_invalid_write_arguments_are_rejected(lib):
    assert _write(lib, k=None) == 1 and _write(lib, v=None) == 1 and _write(lib, slots=None) == 1
    assert _write(lib, n=0) == 2
    assert _write(lib, ks=248) == 2 and _write(lib, vs=257) == 2
    assert _write(lib, k=FAKE + 8) == 3 and _write(lib, v=FAKE + 2) == 3 and _write(lib, slots=FAKE + 2) == 3


def test_invalid_read_arguments_are_rejected(lib):
    assert _read(lib, table=None) == 1 and _read(lib, lens=None) == 1 and _read(lib, k=None) == 1
    assert _read(lib, B=0) == 2 and _read(lib, most=0) == 2 and _read(lib, width=0) == 2
    assert _read(lib, B=1 << 15, most=1 << 20) == 2         # CTAs past 2^31
    assert _read(lib, v=FAKE + 8) == 3 and _read(lib, table=FAKE + 1) == 3 and _read(lib, lens=FAKE + 2) == 3


def test_invalid_attention_arguments_are_rejected(lib):
    assert _attend(lib, q=None) == 1 and _attend(lib, out=None) == 1 and _attend(lib, lens=None) == 1
    assert _attend(lib, B=0) == 2 and _attend(lib, B=8193) == 2 and _attend(lib, T=0) == 2
    assert _attend(lib, Hq=3) == 2 and _attend(lib, Hq=0) == 2 and _attend(lib, width=0) == 2
    assert _attend(lib, qs=504) == 2 and _attend(lib, qs=516) == 2
    assert _attend(lib, width=1 << 28) == 2                 # positions past 2^31
    assert _attend(lib, q=FAKE + 8) == 3 and _attend(lib, out=FAKE + 8) == 3 and _attend(lib, lens=FAKE + 1) == 3
    assert _attend(lib, scale=float("nan")) == 5 and _attend(lib, scale=float("-inf")) == 5
    assert _shared(lib, pp=None) == 1 and _shared(lib, prefix=0) == 2 and _shared(lib, pp=FAKE + 2) == 3
    assert _shared(lib, width=(1 << 27) - 1) == 2
    assert lib.q4_last_error_string() != b""


def test_workspace_bytes_of_invalid_shapes(lib):
    f = lib.q4_kv_attention_workspace_bytes
    assert f(3, 2, 64, 1, 1, 4, 0) == 0 and f(0, 2, 96, 1, 1, 4, 0) == 0
    assert f(0, 2, 64, 0, 1, 4, 0) == 0 and f(0, 2, 64, 1, 1, 3, 0) == 0 and f(0, 2, 64, 1, 1, 4, -1) == 0
