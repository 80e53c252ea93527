"""Float64 definitions of the gated grouped layer (both projections, the activation and their
product) with its gradient, and of the grouped product of 8-bit integers with scales for each
token and channel.  Plain numpy, one group at a time."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc as _erfc

ACTS = ("silu", "gelu", "gelu_tanh")


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _phi(v):
    """The normal distribution (by erfc: 1 + erf cancels where v is negative)."""
    return 0.5 * _erfc(-v / math.sqrt(2.0))


def act(name, v):
    v = np.asarray(v, np.float64)
    if name == "silu":
        return v * _sigmoid(v)
    if name == "gelu":
        return v * _phi(v)
    return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))


def slope(name, v):
    """The activation's derivative."""
    v = np.asarray(v, np.float64)
    if name == "silu":
        s = _sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    if name == "gelu":
        return _phi(v) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * v * v)


def groups(m_splits):
    """(g, rows) of every group: its slice of the packed rows."""
    first = 0
    for g, m in enumerate(m_splits):
        yield g, slice(first, first + int(m))
        first += int(m)


def product(x, w, bias, m_splits):
    """h [T, N] = x W_g^T (+ b_g)."""
    x = np.asarray(x, np.float64)
    h = np.zeros((x.shape[0], np.shape(w[0])[0]))
    for g, r in groups(m_splits):
        h[r] = x[r] @ np.asarray(w[g], np.float64).T + (0.0 if bias is None else np.asarray(bias[g], np.float64))
    return h


def glu(name, h):
    F = h.shape[1] // 2
    return act(name, h[:, :F]) * h[:, F:]


def glu_grad(name, h, da):
    """dh [T, 2F]."""
    F = h.shape[1] // 2
    return np.concatenate([da * h[:, F:] * slope(name, h[:, :F]), da * act(name, h[:, :F])], 1)


def glu_backward(x, w, dh, m_splits):
    """(dx, dw, db) of the layer for the gradient dh of h."""
    x, dh = np.asarray(x, np.float64), np.asarray(dh, np.float64)
    dx, dw, db = np.zeros_like(x), [], []
    for g, r in groups(m_splits):
        dx[r] = dh[r] @ np.asarray(w[g], np.float64)
        dw.append(dh[r].T @ x[r])
        db.append(dh[r].sum(0))
    return dx, np.stack(dw), np.stack(db)


def quantize_int8(x):
    """(codes, scale) of the rows of fp32 (or narrower) values x, every operation rounded to
    fp32 as the definition says."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        m = np.maximum(np.abs(x).max(-1), np.float32(2.0 ** -100)).astype(np.float32)
        good = np.isfinite(x).all(-1)
        inv = (np.float32(127) * (np.float32(1) / m).astype(np.float32)).astype(np.float32)
        q = np.rint((x * inv[..., None]).astype(np.float32))
        q = np.where(good[..., None], q, 0).astype(np.int8)
        scale = np.where(good, (m / np.float32(127)).astype(np.float32), np.float32(np.nan))
    return q, scale


def product_int8(x, x_scale, w, w_scale, bias, m_splits):
    """h [T, N] = (x W_g^T) x_scale[t] w_scale_g[n] (+ b_g)."""
    h = product(x, w, None, m_splits)
    for g, r in groups(m_splits):
        h[r] *= np.asarray(x_scale, np.float64)[r][:, None] * np.asarray(w_scale[g], np.float64)
        if bias is not None:
            h[r] += np.asarray(bias[g], np.float64)
    return h
