"""The distillation loss where everything outside the alternatives lies far below them, against its
definition in 64 bits (logarithms, so that nothing underflows there).

Tolerances.  Loss: means of log probabilities, each off by at most 2e-5 (a sum of up to 2^19 rounded
exponentials, held in 32 bits: 1.4e-5 relative, so absolute in its logarithm; the rest in 64) and one
rounding, 2^-24 of the value; 2^-22 covers it.  A gradient entry is w (q - p - p_t r), r its share
of what lies outside: q and r are off by 4e-5 of themselves (an exponential whose argument, below
127 in units of log 2, carries four roundings, difference, product and two of the constant: 4 * 127 ln 2
2^-24 = 2.1e-5, and the sum's 1.4e-5), then one rounding to the output's type.  An exponential below 2^-126 of the row's (or the outside's) greatest is
taken as 0: |w| 2^-125.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import vocab_tail_ref as ref
from speculative_decode_amd import _lib as L
from speculative_decode_amd import topk_distill, topk_distill_grad

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    L.lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def check(z, ids, top, g, T, tail):
    """both forms of the loss with its gradient"""
    zg = z.detach().clone().requires_grad_(True)
    apart = topk_distill(zg, ids, top, temperature=T, tail=tail)
    d_apart, = torch.autograd.grad(apart, zg, g)
    forms = {"one call": topk_distill_grad(z, ids, top, g, temperature=T, tail=tail), "apart": (apart, d_apart)}
    zz, ii, ll, gg, T32 = f64(z), ids.cpu().numpy(), f64(top), f64(g), float(np.float32(T))
    half = torch.finfo(z.dtype).eps / 2
    for r in range(len(zz)):
        loss, grad, size = ref.distill(zz[r], T32, ii[r], ll[r], tail)
        for name, (l, d) in forms.items():
            got = float(l.detach()[r])
            assert abs(got - loss) <= 2e-5 + 2.0 ** -22 * abs(loss), (name, r, got, loss)
            want = gg[r] * grad
            err = np.abs(f64(d[r]) - want)
            tol = half * np.abs(want) + 4e-5 * abs(gg[r]) * size + abs(gg[r]) / T32 * 2.0 ** -125
            assert (err <= tol).all(), (name, r, np.argwhere(~(err <= tol))[:3], f64(d[r])[~(err <= tol)][:3],
                                        want[~(err <= tol)][:3])


def rows_below(dt, V, k, gap, spread, gen):
    """Four rows: plain, with masked tokens, with alternatives all over the row, with both.  Alternatives
    hold 0.6 of the teacher."""
    z = torch.randn(4, V, generator=gen, device="cuda") / 2 - gap
    ids = torch.empty(4, k, dtype=torch.int32, device="cuda")
    ids[:2] = torch.arange(V // 3, V // 3 + k, device="cuda")          # one beside the other
    ids[2:] = torch.linspace(0, V - 1, k, device="cuda").to(torch.int32)
    mask = torch.rand(4, V, generator=gen, device="cuda") < 0.3
    mask[::2] = False
    z[mask] = -float("inf")
    z.scatter_(1, ids.long(), torch.randn(4, k, generator=gen, device="cuda") * spread)
    p = torch.rand(4, k, generator=gen, device="cuda") + 0.1
    top = torch.log(0.6 * p / p.sum(1, keepdim=True))
    return z.to(dt), ids, top


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [1003, 8000, 70001, 128256])
@pytest.mark.parametrize("gap,T", [(50, 1.0), (79, 1.0), (86, 1.0), (88, 1.0), (90, 1.0), (100, 1.0), (150, 1.0), (700, 1.0),
                                   (10000, 1.0), (5, 0.1), (8.5, 0.1), (10, 0.1), (20, 0.1), (0.5, 1e-4)])
def test_far_below(dt, V, gap, T):
    """rows of one slice and of many, held whole and not, with the gradient of a scaled loss as well"""
    gen = torch.Generator(device="cuda").manual_seed(V + int(gap))
    z, ids, top = rows_below(dt, V, 9, gap, min(0.5, T), gen)
    for scale in (1.0, 65536.0):
        check(z, ids, top, scale * (torch.rand(4, generator=gen, device="cuda") + 0.5), T, True)
    check(z, ids, top, torch.ones(4, device="cuda"), T, False)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [3001, 8000, 70001])
def test_alternatives_far_below(dt, V):
    """the other way round: the student gives the alternatives next to nothing"""
    gen = torch.Generator(device="cuda").manual_seed(V)
    for gap in (60, 88, 200, 5000):
        z, ids, top = rows_below(dt, V, 9, -gap, 0.5, gen)
        for tail in (False, True):
            check(z, ids, top, torch.rand(4, generator=gen, device="cuda") + 0.5, 1.0, tail)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [3001, 8000, 70001])
def test_lowest_value_is_a_number(dt, V):
    """logits of the type's lowest value are numbers, however small their probability: the loss counts what
    the teacher holds there, and its gradient raises them; -inf alone is a mask"""
    gen = torch.Generator(device="cuda").manual_seed(V)
    z, ids, top = rows_below(dt, V, 9, 0, 0.5, gen)
    hot = torch.zeros(4, V, device="cuda").scatter_(1, ids.long(), 1.0) > 0
    z[~hot & torch.isfinite(z)] = torch.finfo(dt).min
    check(z, ids, top, torch.ones(4, device="cuda"), 2.0, True)
    check(z, ids, top, torch.ones(4, device="cuda"), 2.0, False)
    z[~hot] = -float("inf")  # nothing outside
    check(z, ids, top, torch.ones(4, device="cuda"), 2.0, True)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [3001, 8000, 70001])
@pytest.mark.parametrize("where", ["alternative", "outside"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_no_numbers_reach_the_whole_row(dt, V, where, what):
    """one NaN or +inf makes loss and gradient of its row NaN, also where everything else outside the
    alternatives is masked; other rows do not notice"""
    gen = torch.Generator(device="cuda").manual_seed(V)
    z, ids, top = rows_below(dt, V, 9, 3, 0.5, gen)
    z[1, ids[1, 4].long() if where == "alternative" else 2] = what
    hot = torch.zeros(4, V, device="cuda").scatter_(1, ids.long(), 1.0) > 0
    z[2, ~hot[2]] = -float("inf")
    z[2, ids[2, 4].long() if where == "alternative" else 2] = what
    g = torch.ones(4, device="cuda")
    for tail in (False, True):
        zg = z.clone().requires_grad_(True)
        apart = topk_distill(zg, ids, top, tail=tail)
        for loss, d in (topk_distill_grad(z, ids, top, g, tail=tail), (apart, torch.autograd.grad(apart, zg, g)[0])):
            assert torch.isnan(loss[1:3]).all() and torch.isnan(d[1:3].float()).all()
            assert torch.isfinite(loss[[0, 3]]).all() and torch.isfinite(d[[0, 3]].float()).all()
