"""What operands of two and of three bf16 parts cost the states and dA, against the bound that the
GPU tests hold them to (CPU only)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_chunk_ref
import scan_ref

SHAPES = [(1, 200, 16, 64, 64, 2), (2, 150, 8, 128, 128, 2), (1, 150, 8, 64, 256, 1)]


def inputs(b, T, H, P, N, G):
    r = np.random.default_rng(3)
    bf = lambda v: torch.tensor(v, dtype=torch.float32).bfloat16().double().numpy()  # noqa: E731
    f = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    v = dict(x=bf(r.normal(size=(b, T, H, P))), B=bf(r.normal(size=(b, T, G, N)) / 2),
             C=bf(r.normal(size=(b, T, G, N)) / 2), dt=bf(np.log1p(np.exp(r.normal(size=(b, T, H)) - 2))),
             A=f(-np.exp(r.uniform(-6, 0, size=H))), D=f(r.normal(size=H)), h0=f(r.normal(size=(b, H, N, P))))
    return v, bf(r.normal(size=(b, T, H, P))), f(r.normal(size=(b, H, N, P)))


def off(got, want, k):
    return np.linalg.norm(got[k] - want[k]) / np.linalg.norm(want[k])


@pytest.mark.parametrize("shape", SHAPES)
def test_the_bound_tells_two_parts_from_three(shape):
    v, dy, dh = inputs(*shape)
    want = scan_ref.scan(**v, dy=dy, dhT=dh)
    exact = scan_chunk_ref.chunked(**v, dy=dy, dhT=dh)
    two = scan_chunk_ref.chunked(**v, dy=dy, dhT=dh, rounded=scan_chunk_ref.parts(2))
    three = scan_chunk_ref.chunked(**v, dy=dy, dhT=dh, rounded=scan_chunk_ref.parts(3))
    plain = scan_chunk_ref.in_32_bits(**v, dy=dy, dhT=dh)
    for k in ("h", "dh0", "dA"):
        bound = 2 * off(plain, want, k)
        assert off(exact, want, k) < 1e-13 and off(three, want, k) < bound / 10 and off(two, want, k) > 1.5 * bound, k
