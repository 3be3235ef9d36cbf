"""What the gradients of the scan keep of small terms beside large ones, and how far its outputs are
from the 64-bit recurrence as a whole."""
from __future__ import annotations

import pytest
import torch

from speculative_decode_amd import _lib as L
from test_gpu_scan import BF, F32, check, make

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
