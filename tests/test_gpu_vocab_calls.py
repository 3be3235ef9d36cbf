"""Calls of the operators over logits that concern their memory rather than their numbers."""
from __future__ import annotations

import pytest
import torch

from speculative_decode_amd import _lib as L
from speculative_decode_amd import token_logprobs, topk_distill, topk_distill_grad

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    L.lib()


def inputs(rows=4, V=1000, k=5, dt=F32):
    gen = torch.Generator(device="cuda").manual_seed(rows + V)
    z = torch.randn(rows, V, generator=gen, device="cuda").to(dt)
    _, _, ids, top = token_logprobs(torch.randn(rows, V, generator=gen, device="cuda"), top_k=k)
    return z, ids, top, torch.rand(rows, generator=gen, device="cuda")


def test_logits_overwritten_in_place_are_noticed():
    """a graph that has kept the logits must not go on with the gradient in their place"""
    z, ids, top, g = inputs()
    leaf = z.clone().requires_grad_(True)
    soft = torch.tanh(leaf)  # keeps its own result for its gradient
    topk_distill_grad(soft.detach(), ids, top, g, out=soft.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        soft.sum().backward()
    leaf = z.clone().requires_grad_(True)
    loss = topk_distill(leaf, ids, top)
    topk_distill_grad(z, ids, top, g, out=leaf.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    # a result of the call's own making, and the logits' old values elsewhere, are no such thing
    soft = torch.tanh(leaf)
    topk_distill_grad(soft.detach(), ids, top, g)
    topk_distill_grad(soft.detach(), ids, top, g, out=torch.empty_like(z))
    soft.sum().backward()
    with torch.inference_mode():
        out = torch.empty_like(z)
    topk_distill_grad(z, ids, top, g, out=out)


@pytest.mark.parametrize("rows,V", [(1, 2 ** 32 + 5), (2 ** 32 + 3, 1), (2 ** 31, 2)])
def test_sizes_past_32_bits_are_refused(rows, V):
    """not taken for what their lower 32 bits say"""
    z = torch.empty(rows, V, dtype=BF, device="cuda")
    with pytest.raises(L.MilError) as e:
        token_logprobs(z, top_k=1)
    assert e.value.status == L.MIL_E_UNSUPPORTED
    few = torch.zeros(1, 1, dtype=torch.int32, device="cuda").expand(rows, 1)
    with pytest.raises(L.MilError) as e:
        topk_distill(z, few, few.float())
    assert e.value.status == L.MIL_E_UNSUPPORTED


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [1000, 999])
def test_gradient_beside_the_logits(dt, V):
    """logits and gradient as the two halves of each row of one buffer"""
    z, ids, top, g = inputs(V=V, dt=dt)
    want = topk_distill_grad(z, ids, top, g)
    wide = torch.zeros(4, 2 * V, dtype=dt, device="cuda")
    wide[:, :V] = z
    loss, d = topk_distill_grad(wide[:, :V], ids, top, g, out=wide[:, V:])
    assert torch.equal(wide[:, :V], z) and torch.equal(wide[:, V:], d)
    # (an odd row's other half begins off a 16-byte boundary, where the separate launches add up in another order)
    assert (loss - want[0]).abs().max() <= 4e-5
    assert (d.float() - want[1].float()).abs().max() <= 2 * torch.finfo(dt).eps * want[1].float().abs().max() + 1e-6
