"""The layer over whole sequences as a differentiable function (`ssm_scan`): what distilling
attention into it trains.  Marshalling and checks only; the work is in the HIP library
(mil_ssm_scan_forward and mil_ssm_scan_backward)."""
from __future__ import annotations

import ctypes

import torch

from . import _lib as L
from .distill import addr, on_device, stream, workspace
from .ssm import _DTYPES


def _aligned(t):
    """The kernels take tensors on 16-byte boundaries; one that begins between them (a slice of
    a larger buffer) is copied."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, B, C, dt, A, D, h0, lengths, keep):
        x, B, C = _aligned(x), _aligned(B), _aligned(C)
        nseq, T, H, P = x.shape
        dims = L.Dims(nseq, H, P, B.shape[3], B.shape[2])
        code, dev = _DTYPES[x.dtype], x.device
        y = torch.empty_like(x)
        h = torch.empty((nseq, H, B.shape[3], P), dtype=torch.float32, device=dev)
        with on_device(dev):
            flags = 0 if keep else L.MIL_SCAN_FORWARD_ONLY
            need = int(L.lib().mil_ssm_scan_states_bytes(ctypes.byref(dims), T, code, flags))
            states, sp, sb = workspace(need, dev)
            L.check(L.lib().mil_ssm_scan_forward(ctypes.byref(dims), T, code, addr(lengths), addr(x), addr(B),
                                                 addr(C), addr(dt), addr(A), addr(D), addr(h0), addr(y), addr(h),
                                                 sp, sb, flags, stream(dev)), "mil_ssm_scan_forward")
        ctx.set_materialize_grads(False)
        if keep:
            ctx.save_for_backward(x, B, C, dt, A, D, lengths, states)
            ctx.has_h0 = h0 is not None
        return y, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh):
        x, B, C, dt, A, D, lengths, states = ctx.saved_tensors
        nseq, T, H, P = x.shape
        dims = L.Dims(nseq, H, P, B.shape[3], B.shape[2])
        code, dev = _DTYPES[x.dtype], x.device
        dy = torch.zeros_like(x) if dy is None else _aligned(dy.to(x.dtype).contiguous())
        dh = None if dh is None else dh.to(torch.float32).contiguous()
        dx, dB, dC, ddt = (torch.empty_like(t) for t in (x, B, C, dt))
        dA, dD = torch.empty_like(A), torch.empty_like(D)
        dh0 = torch.empty((nseq, H, B.shape[3], P), dtype=torch.float32, device=dev) if ctx.has_h0 else None
        with on_device(dev):
            need = int(L.lib().mil_ssm_scan_workspace_bytes(ctypes.byref(dims), T, code))
            own, ws, ws_bytes = workspace(need, dev)
            sp = (states.data_ptr() + 255) // 256 * 256
            L.check(L.lib().mil_ssm_scan_backward(ctypes.byref(dims), T, code, addr(lengths), addr(x), addr(B),
                                                  addr(C), addr(dt), addr(A), addr(D), sp,
                                                  states.numel() - (sp - states.data_ptr()), addr(dy), addr(dh),
                                                  addr(dx), addr(dB), addr(dC), addr(ddt), addr(dA), addr(dD),
                                                  addr(dh0), ws, ws_bytes, stream(dev)), "mil_ssm_scan_backward")
        return dx, dB, dC, ddt, dA, dD, dh0, None, None


def ssm_scan(x, B, C, dt, A, D, h0=None, lengths=None):
    """h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t^T,  y_t = C_t^T h_t + D x_t over whole
    sequences, differentiable in every floating argument.

    x [nseq][T][H][P], B and C [nseq][T][G][N], dt [nseq][T][H] (float32 or bfloat16, one type);
    A, D [H] float32; h0 [nseq][H][N][P] float32 or None (zeros); lengths [nseq] int32 on
    the device or None: tokens behind a sequence's length are not read, leave its state
    unchanged, and get y and gradients of 0.  Returns (y [nseq][T][H][P] of x's type,
    h_final [nseq][H][N][P] float32).  The inputs must be contiguous."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise ValueError("ssm_scan: x must be [nseq][T][H][P] and B [nseq][T][G][N]")
    if x.device.type != "cuda":
        raise ValueError(f"ssm_scan: tensors must be on a GPU, got {x.device}")
    if x.dtype not in _DTYPES:
        raise TypeError(f"ssm_scan: x must be float32 or bfloat16, got {x.dtype}")
    nseq, T, H, P = (int(n) for n in x.shape)
    G, N = int(B.shape[2]), int(B.shape[3])
    L.check_sizes("ssm_scan", nseq, T, H, P, G, N)
    f32, tok, dev = torch.float32, x.dtype, x.device
    for name, t, shape, dtype in (("x", x, (nseq, T, H, P), tok), ("B", B, (nseq, T, G, N), tok),
                                  ("C", C, (nseq, T, G, N), tok), ("dt", dt, (nseq, T, H), tok), ("A", A, (H,), f32),
                                  ("D", D, (H,), f32), ("h0", h0, (nseq, H, N, P), f32),
                                  ("lengths", lengths, (nseq,), torch.int32)):
        if t is None and name in ("h0", "lengths"):
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev:
            raise TypeError(f"ssm_scan: {name} must be a {dtype} tensor on {dev}")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"ssm_scan: {name} must be a contiguous tensor of shape {shape}, got {tuple(t.shape)}")
    if nseq < 1 or T < 1:
        raise ValueError("ssm_scan: at least one sequence and one token")
    keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, B, C, dt, A, D, h0))
    return _Scan.apply(x, B, C, dt, A, D, h0, lengths, keep)
