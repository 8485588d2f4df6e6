"""Refusals of the attention entry points that come before any launch (fake pointers are never
dereferenced, and no device is asked for)."""
import ctypes

import pytest
import torch

from bit_weight_only_q4_gb300 import build as q4build
from bit_weight_only_q4_gb300 import q4

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load()


def shared(lib, heads, width, page=16, prefix=20, D=128):
    return lib.q4_kv_attention_shared(FAKE, heads * D, FAKE, 0, 4, page, heads, D, FAKE, prefix, FAKE, width, FAKE, 1, 1,
                                      heads, ctypes.c_float(0.1), FAKE, None, 0, None)


def single(lib, heads, width, page=16, D=128):
    return lib.q4_kv_attention(FAKE, heads * D, FAKE, 0, 4, page, heads, D, FAKE, width, FAKE, 1, 1, heads,
                               ctypes.c_float(0.1), FAKE, None, 0, None)


def test_tables_of_too_many_tiles_are_refused_before_the_first_launch(lib):
    """128 tokens a tile: (capacity / 128 + 1) * kv_heads has to stay below 2^31, for the table and the prefix."""
    wide = (1 << 27) - 32                                   # 2^31 - 512 tokens
    assert single(lib, 256, wide) == 2 and shared(lib, 256, wide) == 2
    assert b"kv_heads" in lib.q4_last_error_string()
    assert shared(lib, 256, 1, prefix=(1 << 31) - 1000) == 2
    assert b"kv_heads" in lib.q4_last_error_string()


@pytest.mark.parametrize("page", [0, 8, 24, 2048, 1 << 20, -16])
def test_pages_that_the_calls_refuse_are_not_allocated(page):
    with pytest.raises(ValueError):
        q4.alloc_kv_cache(q4.CACHE_INT8, 4, page, 2, 64, device="cpu")


@pytest.mark.parametrize("shape", [(4,), (4, 2), (4, 2, 1), (4, 2, 1, 2112, 1)])
def test_a_cache_of_other_dimensions_is_a_value_error(monkeypatch, shape):
    monkeypatch.setattr(q4, "_kv_ints", lambda t, name, dims: t.shape)
    with pytest.raises(ValueError, match="cache"):
        q4.q4_kv_attention_shared(torch.zeros(1, 1, 4, 64), torch.zeros(shape, dtype=torch.uint8), torch.zeros(3), 40,
                                  torch.zeros(1, 2), torch.zeros(1), 0)
