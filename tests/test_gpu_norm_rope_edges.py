"""Norms and rotation (q4_norm_rope) where a frequency, a position, a row or eps is at the end of its range."""
from __future__ import annotations

import pytest
import torch

from bit_weight_only_q4_gb300 import q4
from tests.test_gpu_norm_rope import check, made

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
