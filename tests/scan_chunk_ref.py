"""The differentiable scan chunk by chunk in 64 bits, with the operands that are formed on the way
rounded as a caller says, and token by token in 32 bits (numpy): what a given rounding does to the
states and to the gradient of A."""
from __future__ import annotations

import numpy as np

Q = 64


def parts(n):
    """A value as n bf16 numbers that add up to it, as far as they reach"""
    def split(v):
        rest, out = np.asarray(v, dtype=np.float32), np.zeros(np.shape(v))
        for _ in range(n):
            bits = rest.view(np.uint32).astype(np.uint64)
            hi = (((bits + 0x7FFF + ((bits >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)
            out += hi
            rest = rest - hi
        return out
    return split


def chunked(x, B, C, dt, A, D, h0, dy, dhT, rounded=lambda v: v):
    """h, dh0 and dA.  `rounded` is applied to the state, its gradient and weighted tokens where a product
    takes them."""
    b, T, H, P = x.shape
    R = H // B.shape[2]
    out = {"h": np.zeros_like(h0), "dh0": np.zeros_like(h0), "dA": np.zeros(H)}
    for q in range(b):
        for h in range(H):
            g = h // R
            st, states = h0[q, h], []
            cuts = [slice(c, min(T, c + Q)) for c in range(0, T, Q)]
            for s in cuts:
                states.append(st)
                a = np.cumsum(dt[q, s, h] * A[h])
                w = (dt[q, s, h] * np.exp(a[-1] - a))[:, None]
                st = np.exp(a[-1]) * st + rounded(B[q, s, g] * w).T @ x[q, s, h]
            out["h"][q, h] = st
            lam = dhT[q, h]
            for s, st in zip(reversed(cuts), reversed(states)):
                d, Bs, Cs, xs, ys = dt[q, s, h], B[q, s, g], C[q, s, g], x[q, s, h], dy[q, s, h]
                a = np.cumsum(d * A[h])
                low = np.tril(np.ones((len(a), len(a))))
                W = np.exp(np.where(low > 0, a[:, None] - a[None], -np.inf)) * (Cs @ Bs.T) * (ys @ xs.T) * d[None]
                E = np.exp(a) * (Cs * (ys @ rounded(st).T)).sum(1)
                F = np.exp(a[-1] - a) * (Bs * (xs @ rounded(lam).T)).sum(1) * d
                before = np.cumsum(W, 1) - W
                e = (before * low).sum(0) + np.cumsum(E[::-1])[::-1] + np.cumsum(F) - F + np.exp(a[-1]) * (lam * st).sum()
                out["dA"][h] += d @ e
                lam = np.exp(a[-1]) * lam + rounded(Cs * np.exp(a)[:, None]).T @ ys
            out["dh0"][q, h] = lam
    return out


def in_32_bits(x, B, C, dt, A, D, h0, dy, dhT):
    """the same by the recurrence, every operation in fp32"""
    f = np.float32
    x, B, C, dt, A, h0, dy, dhT = (v.astype(f) for v in (x, B, C, dt, A, h0, dy, dhT))
    b, T, H, P = x.shape
    R = H // B.shape[2]
    out = {"h": np.zeros_like(h0), "dh0": np.zeros_like(h0), "dA": np.zeros(H)}
    for q in range(b):
        for h in range(H):
            g, st = h // R, [h0[q, h]]
            dec = np.exp(dt[q, :, h] * A[h])
            for t in range(T):
                st.append(dec[t] * st[-1] + np.outer(dt[q, t, h] * B[q, t, g], x[q, t, h]))
            lam, dA = dhT[q, h], f(0)
            for t in reversed(range(T)):
                lam = dec[t] * (lam + np.outer(C[q, t, g], dy[q, t, h]))
                dA += dt[q, t, h] * np.sum(lam * st[t])
            out["h"][q, h], out["dh0"][q, h] = st[-1], lam
            out["dA"][h] += dA
    return out
