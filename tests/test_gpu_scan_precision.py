"""What the gradients of the scan keep of small terms beside large ones, and how far its outputs are
from the 64-bit recurrence as a whole."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import scan_chunk_ref
import scan_ref
from speculative_decode_amd import _lib as L
from test_gpu_scan import BF, F32, check, f64, make, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    L.lib()


@pytest.mark.parametrize("dt_", [F32, BF])
@pytest.mark.parametrize("P,N", [(16, 16), (64, 64), (128, 128), (64, 256)])
@pytest.mark.parametrize("T", [2, 40, 64, 150])
def test_a_large_last_token(dt_, P, N, T):
    """The exponent's gradient at a token holds nothing of that token's own input, only of what came
    before; a last token of 2^27 is in no other exponent's.  dA is then as exact as without it (the
    bounds of `check`, which are sums of the magnitudes of the terms)."""
    v, dy, dh = make(dt_, 2, T, 4, P, N, 2, seed=T, carry=True, slow=True)
    v["x"][:, -1] *= 2.0 ** 27
    check(v, dy, dh)


SLOW = [(1, 200, 16, 64, 64, 2), (2, 150, 8, 128, 128, 2), (1, 150, 8, 64, 256, 1)]


@pytest.mark.parametrize("shape", SLOW)
def test_states_and_dA_are_those_of_32_bits(shape):
    """bf16 tokens, long memories: the last state, dh0 and dA, each as a whole, are no further from the
    64-bit recurrence than twice what the recurrence in fp32 is, which rounds a state three times a
    token (the kernel: a few times a chunk).  Operands in two bf16 parts instead of three would be
    past it (test_scan_chunk_ref.py)."""
    v, dy, dh = make(BF, *shape, seed=3, carry=True, slow=True)
    got = step(v, dy, dh)
    a = {k: f64(t) for k, t in v.items()}
    want = scan_ref.scan(**a, dy=f64(dy), dhT=f64(dh))
    plain = scan_chunk_ref.in_32_bits(**a, dy=f64(dy), dhT=f64(dh))
    for k in ("h", "dh0", "dA"):
        err, bound = np.linalg.norm(f64(got[k]) - want[k]), 2 * np.linalg.norm(plain[k] - want[k])
        assert err <= bound, (k, err / bound)


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("shape", SLOW + [(2, 70, 8, 32, 32, 1), (3, 20, 8, 128, 128, 2), (4, 1, 8, 32, 64, 1)])
def test_y_and_dx_are_rounded_once(shape, slow):
    """bf16 tokens: y and dx, each as a whole, are as far from the exact values as those rounded to bf16 are.
    What is rounded on the way keeps 16 bits and more (2^-17 of a term at most, against 2^-9 for the
    output), so 5 % of room is plenty; a term rounded to bf16 would take sqrt 2 where the states outweigh the
    tokens, as after a few tokens from a given state."""
    v, dy, dh = make(BF, *shape, seed=13, carry=True, slow=slow)
    got = step(v, dy, dh)
    want = scan_ref.scan(**{k: f64(t) for k, t in v.items()}, dy=f64(dy), dhT=f64(dh))
    for k in ("y", "dx"):
        once = f64(torch.tensor(want[k]).to(BF))
        err, one = np.linalg.norm(f64(got[k]) - want[k]), np.linalg.norm(once - want[k])
        assert err <= 1.05 * one, (k, err / one)
