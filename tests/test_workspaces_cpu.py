"""Which workspaces the binding supplies, and which of them it may let go: the bookkeeping, with
host tensors and a capture that is only said to be one."""
from __future__ import annotations

import contextlib
import gc
import weakref

import pytest
import torch

from bit_weight_only_q4_gb300 import q4

CPU = torch.device("cpu")


@pytest.fixture
def capture(monkeypatch):
    """A list whose first entry is the capture under way (0: none)."""
    now = [0]
    monkeypatch.setattr(q4, "_capture_id", lambda handle, stream: now[0])
    for name in ("_ws_cache", "_ws_held", "_ws_graph", "_kv_ws"):
        monkeypatch.setattr(q4, name, {})
    return now


def attend(n, handle=7):
    return q4._kv_workspace(n, CPU, handle, None)


def test_attention_calls_of_every_shape_share_one(capture):
    a = attend(100_000)
    assert a.numel() == 100_000 and not a[:q4.KV_COUNTER_BYTES].any()
    assert attend(5_000) is a and attend(100_000) is a
    assert attend(100, handle=8) is not a
    b = attend(100_001)
    assert b.numel() >= 200_000 and attend(150_000) is b and attend(1) is b


def test_what_a_capture_was_given_is_never_freed(capture):
    a = weakref.ref(attend(10_000))
    b = weakref.ref(attend(30_000))
    gc.collect()
    assert a() is None                                      # outgrown, and no graph has it
    capture[0] = 3
    assert attend(20_000) is b()
    capture[0] = 0
    for n in range(5):
        attend(50_000 << n)
    for handle in range(100, 200):                          # other streams
        attend(1_000, handle)
    gc.collect()
    assert b() is not None


def test_a_capture_that_comes_first_has_one_of_its_own(capture):
    capture[0] = 5
    a = attend(10_000)
    assert attend(9_000) is a
    larger = attend(11_000)
    assert larger is not a and attend(10_000) is larger
    capture[0] = 0
    eager = attend(10_000)
    assert eager is not a and eager is not larger
    capture[0] = 6
    assert attend(10_000) is eager
    other = attend(12_000)
    assert other is not larger and other is not eager       # another graph's


def project(M, stream=9):
    return q4._default_workspace(q4.LAYOUT_INT4G128, M, 2048, 2048, CPU, stream, stream)


@pytest.fixture
def linear(capture, monkeypatch):
    monkeypatch.setattr(q4, "workspace_bytes", lambda layout, M, N, K: 64 * M)
    monkeypatch.setattr(q4, "_on", lambda stream: contextlib.nullcontext())
    return capture


def test_a_linear_call_keeps_what_its_capture_was_given(linear):
    a = weakref.ref(project(1))
    linear[0] = 4
    assert project(1) is a()
    linear[0] = 0
    for M in range(2, 200):
        project(M)
    gc.collect()
    assert a() is not None


def test_a_linear_call_captured_first_leaves_nothing_to_eager_calls(linear):
    linear[0] = 4
    a = project(3)
    assert project(3) is a
    linear[0] = 0
    assert project(3) is not a                              # its fill has not run


def test_a_workspace_is_filled_on_the_call_s_stream(linear, monkeypatch):
    inside = []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.append(None)

    monkeypatch.setattr(q4, "_on", on)
    project(5, 77)
    assert inside == [77, None]
