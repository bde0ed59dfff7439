"""fp64 CPU reference of the gated feed-forward block, its gradients, the permutation's gradient and clipping.

Plain numpy from the formulas; shares no code with the GPU path.  Beside each output stands what its value
may be off by when the sums behind it are off by given amounts (see the tests' tolerances).
"""
from __future__ import annotations

import math

import numpy as np

from .operators import activation


def spans(offsets, groups, M):
    """(group, first row, end) of the groups that have rows."""
    if offsets is None:
        return [(0, 0, M)] if M else []
    o = np.asarray(offsets, dtype=np.int64)
    return [(e, int(o[e]), int(o[e + 1])) for e in range(groups) if o[e + 1] > o[e]]


def gate_up(x, w1, w3, act):
    """(h, g, u) of one group's rows in fp64."""
    g, u = x @ w1.T, x @ w3.T
    return activation(g, act)[0] * u, g, u


def backward(dy, x, g, u, h, w1, w3, w2, act):
    """dict of one group's gradients in fp64, with the values on the way (dh, dg, du)."""
    value, slope = activation(g, act)
    dh = dy @ w2
    dg, du = dh * u * slope, dh * value
    return {"dh": dh, "dg": dg, "du": du, "dx": dg @ w1 + du @ w3, "dw1": dg.T @ x, "dw3": du.T @ x, "dw2": dy.T @ h}


def permute_backward(dx_perm, slot_to_row, addend, T, top_k, n_shared):
    """(dx, sum of sizes of the terms) in fp64."""
    d = dx_perm.shape[1]
    dx = np.zeros((T, d)) if addend is None else np.array(addend, dtype=np.float64)
    size = np.abs(dx)
    for t in range(T):
        slots = [t * top_k + j for j in range(top_k)] + ([T * top_k + t] if n_shared else [])
        for s in slots:
            r = int(slot_to_row[s])
            if r >= 0:
                dx[t] += dx_perm[r]
                size[t] += np.abs(dx_perm[r])
    return dx, size


def clip(grads, max_norm):
    """(sum of squares, norm, scaled gradients) in fp64; nothing is scaled by a norm that fp32 does not hold."""
    total = math.fsum(float(np.dot(g.ravel(), g.ravel())) for g in grads)
    norm = math.sqrt(total)
    fits = norm < 2.0 ** 128 - 2.0 ** 103                     # rounds to FLT_MAX or less
    scale = max_norm / norm if norm > max_norm and fits else 1.0
    return total, norm, [g * scale for g in grads]
