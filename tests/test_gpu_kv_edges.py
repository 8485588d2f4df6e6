"""The key/value cache and its attention at the edges: inputs, shapes and ways of calling that
test_gpu_kv_cache.py does not reach.  Its helpers and its bound (see there) are used throughout."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import kv_reference as R
from tests.test_gpu_kv_cache import FMTS, bf16, bits, call, filled, q4  # noqa: F401

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
