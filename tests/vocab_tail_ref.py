"""The distillation loss of one row in 64 bits with logarithms instead of probabilities, so that
what lies outside the alternatives is right however far below them it is."""
from __future__ import annotations

import numpy as np


def logsumexp(v):
    m = v.max(initial=-np.inf)
    return m if m == -np.inf else m + np.log(np.exp(v - m).sum())


def distill(z, T, ids, lps, tail):
    """(loss, dloss/dz, the sum of the absolute values of what each gradient entry subtracts); the
    row's logits hold no NaN and no +inf, and not all of them are masked"""
    z = np.asarray(z, dtype=np.float64) / T
    p, hot = np.zeros(len(z)), np.zeros(len(z), dtype=bool)
    for i, l in zip(ids, lps):
        if i >= 0:
            p[i] += np.exp(float(l))
            hot[i] = True
    mass = p.sum()
    lse = logsumexp(z)
    lq, out = z - lse, logsumexp(z[~hot])
    q = np.exp(lq)
    if not tail:
        p = p / mass
    on = p > 0
    loss = (p[on] * (np.log(p[on]) - lq[on])).sum()
    outside = np.zeros(len(z))
    pt = max(0.0, 1 - mass)
    if tail and out > -np.inf:
        if pt > 0:
            loss += pt * (np.log(pt) - (out - lse))
        # (not e^(z - out): at the type's lowest value the logarithm of a count is lost in `out`)
        r = np.exp(z[~hot] - z[~hot].max())
        outside[~hot] = pt * r / r.sum()
    return loss, (q - p - outside) / T, (q + p + outside) / T
