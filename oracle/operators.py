"""fp64 CPU reference of the scored router, the dense product and the gate's gradients.

Plain numpy from the formulas; shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np


# ---- scored routing ----

def scores(logits: np.ndarray, kind: str) -> np.ndarray:
    """softmax or sigmoid of the rows in fp64; a row of -inf only has no score."""
    x = np.asarray(logits, dtype=np.float64)
    if kind == "sigmoid":
        e = np.exp(-np.abs(x))
        return np.where(x < 0, e, 1.0) / (1.0 + e)
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    z = e.sum(axis=1, keepdims=True)
    return np.divide(e, z, out=np.zeros_like(e), where=z > 0)


def _normalised(row: np.ndarray, kind: str) -> np.ndarray:
    """Weights over the chosen logits that sum to 1: s / sum(s), from ln s so that underflow does not matter."""
    if np.all(np.isneginf(row)):
        return np.zeros_like(row)
    ln_s = row if kind == "softmax" else -np.logaddexp(0.0, -row)
    e = np.exp(ln_s - ln_s.max())
    return e / e.sum()


def route_scored(logits, balance_bias, top_k, kind="softmax", n_groups=1, topk_groups=1, group_top=1,
                 renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k] fp64, scores [T, E] fp64, next_ids [T, 2])."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    s = scores(x, kind)
    gs = E // n_groups
    ids = np.full((T, top_k), -1, dtype=np.int64)
    nxt = np.full((T, 2), -1, dtype=np.int64)
    w = np.zeros((T, top_k))
    for t in range(T):
        c = x[t] if balance_bias is None else s[t] + np.asarray(balance_bias, dtype=np.float64)
        per_group = c if balance_bias is not None or group_top == 1 else s[t]
        best = []
        for g in range(n_groups):
            top = sorted(per_group[g * gs:(g + 1) * gs], reverse=True)[:group_top]
            best.append((-sum(top), g))
        open_groups = {g for _, g in sorted(best)[:topk_groups]}
        order = sorted((-c[e], e) for e in range(E) if e // gs in open_groups)
        chosen = [e for _, e in order]
        ids[t] = chosen[:top_k]
        for j, e in enumerate(chosen[top_k:top_k + 2]):
            nxt[t, j] = e
        kept = x[t, ids[t]]
        w[t] = scale * (_normalised(kept, kind) if renormalize else s[t, ids[t]])
    return ids, w, s, nxt


def route_scored_backward(logits, ids, dweights, dscores, kind="softmax", renormalize=True, scale=1.0):
    """Gradient at the logits: the Jacobians of the weights and of the scores, row by row."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    s = scores(x, kind)
    out = np.zeros((T, E))
    for t in range(T):
        jac = np.diag(s[t]) - np.outer(s[t], s[t]) if kind == "softmax" else np.diag(s[t] * scores(-x[t:t + 1], kind)[0])
        if dscores is not None:
            out[t] += np.asarray(dscores[t], dtype=np.float64) @ jac
        e = np.asarray(ids[t], dtype=np.int64)
        g = scale * np.asarray(dweights[t], dtype=np.float64)
        if renormalize:
            v = _normalised(x[t, e], kind)
            dln = (np.diag(v) - np.outer(v, v)) @ g           # gradient at ln s of the chosen
            out[t, e] += dln if kind == "softmax" else dln * scores(-x[t:t + 1, e], kind)[0]
        else:
            out[t] += g @ jac[e]
    return out


# ---- combine ----

def combine_backward(dy, y_perm, slot_to_row, weights, top_k, n_shared):
    """({row: gradient}, dweights [T, k])."""
    dy = np.asarray(dy, dtype=np.float64)
    T = dy.shape[0]
    rows, dw = {}, np.zeros((T, top_k))
    for t in range(T):
        for j in range(top_k):
            r = int(slot_to_row[t * top_k + j])
            if r >= 0:
                rows[r] = float(weights[t, j]) * dy[t]
                dw[t, j] = dy[t] @ np.asarray(y_perm[r], dtype=np.float64)
        if n_shared:
            rows[int(slot_to_row[T * top_k + t])] = dy[t]
    return rows, dw


# ---- dense product ----

_erf = np.vectorize(math.erf, otypes=[float])


def activation(p, act):
    """(act(p), act'(p)) in fp64."""
    p = np.asarray(p, dtype=np.float64)
    if act == "none":
        return p, np.ones_like(p)
    if act == "relu":
        return np.maximum(p, 0.0), (p > 0).astype(np.float64)
    if act == "silu":
        sg = scores(p, "sigmoid")
        return p * sg, sg + p * sg * scores(-p, "sigmoid")
    if act == "gelu":
        cdf = 0.5 * (1.0 + _erf(p / math.sqrt(2.0)))
        return p * cdf, cdf + p * np.exp(-0.5 * p * p) / math.sqrt(2.0 * math.pi)
    u = math.sqrt(2.0 / math.pi) * (p + 0.044715 * p ** 3)
    th = np.tanh(u)
    return (0.5 * p * (1.0 + th),
            0.5 * (1.0 + th) + 0.5 * p * (1.0 - th * th) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * p * p))


def linear(x, w, bias, residual, act):
    """(y, pre) in fp64."""
    p = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    if bias is not None:
        p = p + np.asarray(bias, dtype=np.float64)
    y = activation(p, act)[0]
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
    return y, p


def linear_backward(dy, pre, x, w, act):
    """(dx, dw, dbias, dpre) in fp64."""
    d = np.asarray(dy, dtype=np.float64)
    if act != "none":
        d = d * activation(pre, act)[1]
    return d @ np.asarray(w, dtype=np.float64), d.T @ np.asarray(x, dtype=np.float64), d.sum(axis=0), d
