"""Float64 definitions of the operators around the experts: the RMS norm with the
residual's addition, the token routing and the expert layer of a few tokens.  Plain
numpy, one token or row at a time where that is clearest."""
from __future__ import annotations

import numpy as np

from .grouped_mlp import silu


def rmsnorm(x, gamma, eps, residual=None):
    """(h, y): h = x (+ residual), y = h / sqrt(mean(h^2) + eps) * gamma."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    with np.errstate(all="ignore"):
        r = np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
        return h, h / r * np.asarray(gamma, np.float64)


def rmsnorm_backward(dy, h, gamma, eps, dh=None):
    """(dx, dgamma) of the norm at h for the gradient dy of y and dh of h."""
    h, v = np.asarray(h, np.float64), np.asarray(dy, np.float64) * np.asarray(gamma, np.float64)
    r = np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    dx = v / r - h * np.mean(v * h, axis=1, keepdims=True) / r ** 3
    if dh is not None:
        dx = dx + dh
    return dx, np.sum(np.asarray(dy, np.float64) * h / r, axis=0)


def _masked(l):
    """NaN counts as -inf (masked), +inf as the largest finite fp32 value."""
    return np.minimum(np.where(np.isnan(l), -np.inf, l), float(np.finfo(np.float32).max))


def _sigmoid(l):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-l))


def route(logits, top_k, sigmoid=False, renormalize=True):
    """(ids, weights) of every token: the largest logits, ties to the lowest expert, NaN
    as -inf, +inf as the largest finite value; a masked (-inf) expert weighs 0."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    ids, weights = np.zeros((T, top_k), np.int64), np.zeros((T, top_k))
    for t in range(T):
        l = _masked(logits[t])
        chosen = sorted(range(E), key=lambda e: (-l[e], e))[:top_k]
        scores = np.zeros(E)
        live = l > -np.inf
        if sigmoid:
            scores[live] = _sigmoid(l[live])
        elif live.any():
            scores[live] = np.exp(l[live] - l[live].max())
            scores /= scores.sum()
        w = scores[chosen]
        if renormalize and w.sum() > 0:
            w = w / w.sum()
        ids[t], weights[t] = chosen, w
    return ids, weights


def plan(ids, num_experts):
    """(m_splits, row_index, slot_index): slots ordered by expert, then by slot."""
    flat = [int(e) for e in np.asarray(ids).reshape(-1)]
    slots = sorted(range(len(flat)), key=lambda s: (flat[s], s))
    rows = np.zeros(len(flat), np.int64)
    for r, s in enumerate(slots):
        rows[s] = r
    splits = np.array([flat.count(e) for e in range(num_experts)], np.int64)
    return splits, rows.reshape(np.asarray(ids).shape), np.array(slots, np.int64)


def route_backward(logits, ids, dweights, sigmoid=False, renormalize=True):
    """dlogits: the gradient of sum(dweights * weights) with the choice held fixed."""
    logits = np.asarray(logits, np.float64)
    out = np.zeros_like(logits)
    for t in range(logits.shape[0]):
        l = _masked(logits[t])
        live = l > -np.inf
        if not live.any():
            continue
        c = np.asarray(ids[t], np.int64)
        s, d = np.zeros(c.size), np.asarray(dweights[t], np.float64)
        if sigmoid:
            s[live[c]] = _sigmoid(l[c][live[c]])
            if renormalize and s.sum() > 0:  # w = s / sum(s)
                d = (d - d @ s / s.sum()) / s.sum()
            out[t, c] = d * s * (1 - s)
        elif renormalize:  # a softmax over the chosen
            s[live[c]] = np.exp(l[c][live[c]] - l[c].max())
            s /= s.sum()
            out[t, c] = s * (d - d @ s)
        else:
            p = np.zeros_like(l)
            p[live] = np.exp(l[live] - l[live].max())
            p /= p.sum()
            dp = np.zeros_like(l)
            dp[c] = d
            out[t] = p * (dp - dp @ p)
    return out


def moe(x, ids, weights, w1, w2, b1=None, b2=None, residual=None):
    """The expert layer, slot by slot; ids outside the experts take no part."""
    x, w1, w2 = (np.asarray(a, np.float64) for a in (x, w1, w2))
    E, F2, _ = w1.shape
    y = np.zeros((x.shape[0], w2.shape[1])) if residual is None else np.array(residual, np.float64)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0 or e >= E or weights[t, j] == 0:
                continue
            h = w1[e] @ x[t] + (0.0 if b1 is None else b1[e])
            z = w2[e] @ (silu(h[:F2 // 2]) * h[F2 // 2:]) + (0.0 if b2 is None else b2[e])
            y[t] += weights[t, j] * z
    return y
