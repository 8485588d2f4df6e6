"""What the operators around a layer's projections take and refuse at the ends of their ranges, before any launch: 5 is a
refused argument; 6 or 7, no device, that the checks were passed."""
import pytest
import torch

from bit_weight_only_q4_gb300 import build as q4build
from bit_weight_only_q4_gb300 import q4
from tests.test_layer_refusals_cpu import FAKE, INF, lora, prompt, rope

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would be launched")
PASSED = (6, 7)
APART = dict(q=FAKE, qo=FAKE, k=2 * FAKE, ko=2 * FAKE)       # q and k in place, each elsewhere


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load()


@no_gpu
def test_eps(lib):
    for eps in (0.0, 1e-45, 1e-6, 1.0, 1e30):
        assert rope(lib, eps=eps, **APART) in PASSED
    for eps in (1.1e30, 1e37, 3e38, INF, -1e-45):
        assert rope(lib, eps=eps, **APART) == 5


@no_gpu
def test_pointers_of_no_heads_and_of_no_rotation_are_not_looked_at(lib):
    for name in ("q", "qo", "qw"):
        assert rope(lib, Hq=0, **dict(APART, **{name: FAKE + 2})) in PASSED
        assert rope(lib, Hq=0, **dict(APART, **{name: None})) in PASSED
        assert rope(lib, H=0, **dict(APART, **{name: FAKE + 2})) == 3
    for name in ("k", "ko", "kw"):
        assert rope(lib, H=0, **dict(APART, **{name: FAKE + 2})) in PASSED
        assert rope(lib, H=0, **dict(APART, **{name: None})) in PASSED
        assert rope(lib, Hq=0, **dict(APART, **{name: FAKE + 2})) == 3
    for name in ("pos", "freq"):
        assert rope(lib, rotary=0, **dict(APART, **{name: FAKE + 1})) in PASSED
        assert rope(lib, rotary=0, **dict(APART, **{name: None})) in PASSED
        assert rope(lib, **dict(APART, **{name: FAKE + 1})) == 3


@no_gpu
def test_scales_whose_exponents_of_two_are_numbers(lib):
    apart = dict(q=2 * FAKE, k=2 * FAKE, v=2 * FAKE)
    for scale in (0.0, 1e-45, 1.0, 2e38, -2e38):
        assert prompt(lib, scale=scale, **apart) in PASSED
    for scale in (2.4e38, -2.4e38, 3.4e38, INF, float("nan")):
        assert prompt(lib, scale=scale, **apart) == 5
