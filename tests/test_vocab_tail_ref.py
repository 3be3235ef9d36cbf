"""The 64-bit reference of rows whose tokens outside the alternatives lie far below them (CPU only)."""
from __future__ import annotations

import numpy as np
import pytest

import vocab_ref
import vocab_tail_ref as ref


def row(gap, V=40, k=4):
    rng = np.random.default_rng(int(gap))
    z = rng.normal(size=V) - gap
    z[:k] += gap
    return z, list(range(k)), list(np.log(np.full(k, 0.15)))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("gap", [0, 5, 80, 300, 600])
def test_agrees_with_the_plain_reference(gap, tail):
    """as far as e^-gap is a 64-bit number with all its bits"""
    z, ids, lps = row(gap)
    loss, g, _ = ref.distill(z, 1.0, ids, lps, tail)
    want, gw = vocab_ref.distill(z, 1.0, ids, lps, tail)
    assert abs(loss - want) <= 1e-12 * max(1, abs(want)) and np.abs(g - gw).max() <= 1e-12


@pytest.mark.parametrize("gap,T", [(3, 1.0), (100, 1.0), (5000, 1.0), (30, 0.1)])
def test_gradient_against_differences(gap, T):
    z, ids, lps = row(gap)
    z[7] = -np.inf
    _, g, _ = ref.distill(z, T, ids, lps, True)
    assert abs(g.sum()) <= 1e-12 / T and g[7] == 0
    for i in (0, 3, 4, 20, 39):
        e = np.zeros(len(z))
        e[i] = 1e-4 * T
        d = (ref.distill(z + e, T, ids, lps, True)[0] - ref.distill(z - e, T, ids, lps, True)[0]) / (2 * e[i])
        # h^2 = 1e-8 of a third derivative below 1, and rounding: 1e-16 of a loss below 3000, over h
        assert abs(d - g[i]) * T <= 1e-8 + 1e-12 * max(1, gap / T)
