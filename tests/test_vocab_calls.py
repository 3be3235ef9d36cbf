"""Where the gradient of the loss may lie (CPU only: the workspace is missing, so nothing is enqueued)."""
from __future__ import annotations

import ctypes

import pytest

from speculative_decode_amd import _lib as L

FAKE = 0x7F0000000000


def place(elements, ostride, rows=4, V=100, stride=256, dt=1):
    """status of a call whose dlogits begin `elements` behind the logits; MIL_E_WORKSPACE: its place was accepted"""
    p = ctypes.c_void_p
    out = FAKE + elements * (2 if dt else 4)
    return L.lib().mil_ssm_distill_grad(p(FAKE), rows, V, stride, dt, 1.0, p(FAKE), p(FAKE), 3, 0, p(FAKE), p(FAKE),
                                        p(out), ostride, None, 0, None)


@pytest.mark.parametrize("dt", [0, 1])
def test_gradient_between_the_rows_of_the_logits(dt):
    """two halves of one buffer: the rows alternate and do not touch"""
    for at in (100, 128, 156, -100, -156, 256 + 100, 3 * 256 + 156, -3 * 256 - 100):
        assert place(at, 256, dt=dt) == L.MIL_E_WORKSPACE, at
    for at in (1, 99, 157, 255, 256, 512, -1, -99, -256, 3 * 256 - 1):  # rows that do
        assert place(at, 256, dt=dt) == L.MIL_E_INVALID, at
    assert place(0, 256, dt=dt) == L.MIL_E_WORKSPACE
    for at in (0, 128, -200):  # rows at another distance meet sooner or later
        assert place(at, 300, dt=dt) == L.MIL_E_INVALID, at
    for at in (3 * 256 + 100, -3 * 300 - 100):  # apart as a whole
        assert place(at, 300, dt=dt) == L.MIL_E_WORKSPACE, at
    assert place(50, 100, V=100, stride=100) == L.MIL_E_INVALID


def test_rows_too_far_apart_are_refused():
    """addresses that would not fit 64 bits; their arithmetic overflowed in the check of the places"""
    assert place(128, 256, stride=1 << 55) == L.MIL_E_UNSUPPORTED
    assert place(1 << 20, 1 << 55) == L.MIL_E_UNSUPPORTED
    assert place(1 << 20, 256, stride=1 << 54, rows=1) == L.MIL_E_WORKSPACE
