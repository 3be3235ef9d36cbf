"""Operators over rows of vocabulary logits: what a teacher or verifier says about tokens
(`token_logprobs`) and the loss that moves a student towards a teacher's top alternatives
(`topk_distill`, `topk_distill_grad`).

Marshalling and checks only; the work is in the HIP library (mil_ssm_token_logprobs and
mil_ssm_distill_*).  Every call runs on the current stream of the logits' device.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib as L
from .ssm import _DTYPES


def on_device(dev):
    """The kernels of a call run on the tensors' own device, whichever is current."""
    if torch.cuda.current_device() == dev.index:
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def stream(dev):
    """The current stream of a device as ctypes takes it (the Stream object that
    torch.cuda.current_stream makes on the way costs a tenth of a small call)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def addr(t):
    """A tensor's address as ctypes takes it (None: a null pointer)."""
    return None if t is None else t.data_ptr()


def workspace(nbytes, dev):
    """(tensor that owns it, 256-byte aligned address, bytes).  The caching allocator gives out
    aligned blocks; one that does not is asked for more."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    p = t.data_ptr()
    if p % 256:
        t = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
        p = (t.data_ptr() + 255) // 256 * 256
    return t, p, nbytes


def _rows(what, t):
    """(rows, vocab, row stride) of a [..., vocab] tensor whose rows are evenly spaced."""
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise ValueError(f"{what}: logits must be a [..., vocab] tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what}: tensors must be on a GPU, got {t.device}")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{what}: logits must be float32 or bfloat16, got {t.dtype}")
    V = int(t.shape[-1])
    if V < 1:
        raise ValueError(f"{what}: an empty vocabulary")
    L.check_sizes(what, V, t.numel() // V)
    if t.is_contiguous():
        return t.numel() // V, V, V
    lead = [(n, st) for n, st in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    rows = 1
    for n, _ in lead:
        rows *= int(n)
    even = all(a[1] == b[0] * b[1] for a, b in zip(lead, lead[1:]))
    stride = int(lead[-1][1]) if lead else V
    if rows and ((V > 1 and t.stride(-1) != 1) or not even or stride < V):
        raise ValueError(f"{what}: logits must have contiguous rows at an even distance of at least {V} elements")
    return rows, V, max(stride, V)


def _side(what, name, t, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev:
        raise TypeError(f"{what}: {name} must be a {dtype} tensor on {dev}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be a contiguous tensor of shape {tuple(shape)}")


def logprobs_workspace_bytes(rows, vocab, dtype, top_k) -> int:
    return int(L.lib().mil_ssm_logprobs_workspace_bytes(rows, vocab, _DTYPES[dtype], top_k))


def distill_workspace_bytes(rows, vocab, dtype) -> int:
    return int(L.lib().mil_ssm_distill_workspace_bytes(rows, vocab, _DTYPES[dtype]))


def token_logprobs(logits, tokens=None, top_k=0, temperature=1.0, want_entropy=True):
    """Log probabilities of given tokens, entropies and top alternatives of rows of logits
    (mil_ssm_token_logprobs).

    logits [..., V] float32 or bfloat16 (rows evenly spaced: a padded vocabulary's slice
    needs no copy), tokens [...] int32 or None (negative: no token).  Returns (logprob
    [...], entropy [...], top_ids [..., top_k] int32, top_logprobs [..., top_k]), float32,
    with None in the place of what was not asked for.  No gradients are recorded."""
    what = "token_logprobs"
    rows, V, stride = _rows(what, logits)
    dev, lead = logits.device, tuple(logits.shape[:-1])
    if tokens is not None:
        _side(what, "tokens", tokens, lead, torch.int32, dev)
    top_k = int(top_k)
    if not 0 <= top_k <= min(V, L.MIL_TOPK_MAX):
        raise ValueError(f"{what}: top_k must be 0..{min(V, L.MIL_TOPK_MAX)}, got {top_k}")
    new = lambda shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
    lp = new(lead) if tokens is not None else None
    ent = new(lead) if want_entropy else None
    ids, top = (new(lead + (top_k,), torch.int32), new(lead + (top_k,))) if top_k else (None, None)
    with on_device(dev):
        need = logprobs_workspace_bytes(rows, V, logits.dtype, top_k)
        own, ws, ws_bytes = workspace(need, dev)
        L.check(L.lib().mil_ssm_token_logprobs(addr(logits), rows, V, stride, _DTYPES[logits.dtype],
                                               float(temperature), addr(tokens), top_k, addr(lp), addr(ent),
                                               addr(ids), addr(top), ws, ws_bytes, stream(dev)),
                "mil_ssm_token_logprobs")
    return lp, ent, ids, top


def _check_distill(what, logits, top_ids, top_logprobs):
    rows, V, stride = _rows(what, logits)
    dev, lead = logits.device, tuple(logits.shape[:-1])
    if not isinstance(top_ids, torch.Tensor) or top_ids.dim() != logits.dim():
        raise ValueError(f"{what}: top_ids must be an int32 tensor of shape {lead + ('k',)}")
    k = int(top_ids.shape[-1])
    if not 1 <= k <= L.MIL_TOPK_MAX:
        raise ValueError(f"{what}: 1..{L.MIL_TOPK_MAX} alternatives a row, got {k}")
    _side(what, "top_ids", top_ids, lead + (k,), torch.int32, dev)
    _side(what, "top_logprobs", top_logprobs, lead + (k,), torch.float32, dev)
    return rows, V, stride, k, dev, lead


class _TopkDistill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_ids, top_logprobs, temperature, tail):
        rows, V, stride, k, dev, lead = _check_distill("topk_distill", logits, top_ids, top_logprobs)
        loss = torch.empty(lead, dtype=torch.float32, device=dev)
        stats = torch.empty((max(rows, 1), 4), dtype=torch.float32, device=dev)
        flags = L.MIL_DISTILL_TAIL if tail else 0
        code = _DTYPES[logits.dtype]
        with on_device(dev):
            need = distill_workspace_bytes(rows, V, logits.dtype)
            own, ws, ws_bytes = workspace(need, dev)
            L.check(L.lib().mil_ssm_distill_forward(addr(logits), rows, V, stride, code, float(temperature),
                                                    addr(top_ids), addr(top_logprobs), k, flags, addr(loss),
                                                    addr(stats), ws, ws_bytes, stream(dev)),
                    "mil_ssm_distill_forward")
        ctx.save_for_backward(logits, top_ids, top_logprobs, stats)
        ctx.args = (rows, V, stride, k, code, float(temperature), flags)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        logits, top_ids, top_logprobs, stats = ctx.saved_tensors
        rows, V, stride, k, code, temperature, flags = ctx.args
        dev = logits.device
        grad_loss = grad_loss.to(torch.float32).contiguous()
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        with on_device(dev):
            L.check(L.lib().mil_ssm_distill_backward(addr(logits), rows, V, stride, code, temperature, addr(top_ids),
                                                     addr(top_logprobs), k, flags, addr(stats), addr(grad_loss),
                                                     addr(out), V, stream(dev)),
                    "mil_ssm_distill_backward")
        return out, None, None, None, None


def topk_distill(logits, top_ids, top_logprobs, temperature=1.0, tail=True):
    """Distillation loss of rows of student logits against a teacher's top alternatives, as
    `token_logprobs` of the teacher's logits at the same temperature gives them.

    logits [..., V] float32 or bfloat16; top_ids [..., k] int32 (negative: absent),
    top_logprobs [..., k] float32.  Returns the loss per row [...] float32, differentiable in
    logits: KL(p || q) with everything outside the alternatives as one outcome (`tail`), or
    with the teacher's probabilities divided by their sum.  A row with no alternative has
    loss 0 and gradient 0."""
    return _TopkDistill.apply(logits, top_ids, top_logprobs, temperature, bool(tail))


def topk_distill_grad(logits, top_ids, top_logprobs, grad_loss, temperature=1.0, tail=True, out=None):
    """`topk_distill` and its gradient in one call, for a step that knows each row's weight:
    grad_loss [...] float32.  Returns (loss [...], dlogits [..., V]); `out` may supply dlogits
    (rows evenly spaced), and may be the logits themselves, which are then overwritten: as after
    any in-place operation, a backward pass that needs their old values raises.
    No gradients are recorded."""
    what = "topk_distill_grad"
    rows, V, stride, k, dev, lead = _check_distill(what, logits, top_ids, top_logprobs)
    _side(what, "grad_loss", grad_loss, lead, torch.float32, dev)
    given = out is not None
    if not given:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev:
        raise ValueError(f"{what}: out must be a {logits.dtype} tensor of shape {tuple(logits.shape)} on {dev}")
    ostride = _rows(what, out)[2]
    loss = torch.empty(lead, dtype=torch.float32, device=dev)
    code = _DTYPES[logits.dtype]
    with on_device(dev):
        need = distill_workspace_bytes(rows, V, logits.dtype)
        own, ws, ws_bytes = workspace(need, dev)
        L.check(L.lib().mil_ssm_distill_grad(addr(logits), rows, V, stride, code, float(temperature), addr(top_ids),
                                             addr(top_logprobs), k, L.MIL_DISTILL_TAIL if tail else 0,
                                             addr(grad_loss), addr(loss), addr(out), ostride, ws, ws_bytes,
                                             stream(dev)),
                "mil_ssm_distill_grad")
    if given:  # so that a graph that has kept what was overwritten notices
        torch.autograd.graph.increment_version(out)
    return loss, out
