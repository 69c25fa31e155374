"""The draw from a truncated softmax in plain NumPy, fp64, one row at a time: the definition of
fgmm_sample_logits (include/fgmm.h).  Test infrastructure only."""
import math

import numpy as np


def row(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(id, prob, margin): margin is how far the draw's target and the top-p cut are from the next
    decision, in units of the largest weight."""
    x = np.asarray(x, dtype=np.float64)
    ok = t >= 0 and math.isfinite(t) and 0 < p <= 1 and 0 <= m <= 1 and 0 <= u < 1
    if not ok or np.isnan(x).any():
        return -1, math.nan, math.inf
    if not (x > -np.inf).any():
        return -1, 0.0, math.inf
    top = x.max()
    if t == 0:
        return int(np.argmax(x)), 1.0, math.inf
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / t))
    order = np.lexsort((np.arange(len(x)), -x))
    if 0 < k < len(x):
        order = order[:k]
    margin = math.inf
    if p < 1:
        mass = np.cumsum(w[order])
        before = mass - w[order]
        keep = before < p * mass[-1]
        keep[0] = True
        margin = np.min(np.abs(before - p * mass[-1]))
        order = order[keep]
    order = np.sort(order[w[order] >= m])
    mass = np.cumsum(w[order])
    target = u * mass[-1]
    j = min(int(np.searchsorted(mass, target, side="right")), len(order) - 1)
    margin = min(margin, np.min(np.abs(mass[:-1] - target)) if len(mass) > 1 else math.inf)
    return int(order[j]), float(w[order[j]] / mass[-1]), margin


def rows(x, u, t=None, k=None, p=None, m=None):
    def at(v, i, d):
        return d if v is None else (v if np.isscalar(v) else v[i])
    got = [row(x[i], u[i], at(t, i, 1.0), int(at(k, i, 0)), float(at(p, i, 1.0)), float(at(m, i, 0.0)))
           for i in range(len(x))]
    return (np.array([g[0] for g in got], dtype=np.int32), np.array([g[1] for g in got]),
            np.array([g[2] for g in got]))
