"""Calls of the scan that concern its arguments rather than its numbers."""
from __future__ import annotations

import pytest
import torch

from speculative_decode_amd import _lib as L
from speculative_decode_amd import ssm_scan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    L.lib()


@pytest.mark.parametrize("nseq,T", [(1, 2 ** 32 + 1), (2 ** 32 + 1, 1), (1, 2 ** 31)])
def test_sizes_past_32_bits_are_refused(nseq, T):
    """not taken for what their lower 32 bits say (views of one value: what counts is the shape)"""
    one = torch.zeros(1, 1, 1, 1, dtype=torch.bfloat16, device="cuda")
    x = one.expand(nseq, T, 1, 16)
    A = torch.zeros(1, device="cuda")
    with pytest.raises(L.MilError) as e:
        ssm_scan(x, x, x, x[..., 0], A, A)
    assert e.value.status == L.MIL_E_UNSUPPORTED
