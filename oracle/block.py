"""Plain 64-bit NumPy forms of the operators around the token path: the layer
norm, the balance loss and the dense products with their epilogue, and their
gradients.  Test infrastructure only; shares nothing with the CUDA code.
Inputs are float64 arrays (the exact values of the fp32 or bf16 inputs)."""
from __future__ import annotations

import math

import numpy as np


def layernorm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def layernorm_bwd(dy, x, w, mean, rstd, dres=None):
    """(dx, dw, db) from the given statistics."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    return dx, (dy * xh).sum(0), dy.sum(0)


def _softmax(logits):
    """(p, lse).  -inf and fp32's lowest value mask an expert (p = 0); a row
    of nothing else has lse = -inf."""
    logits = np.where(logits <= np.finfo(np.float32).min, -np.inf, logits)
    top = logits.max(-1, keepdims=True)
    base = np.where(np.isneginf(top), 0.0, top)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        ex = np.exp(logits - base)
        tot = ex.sum(-1, keepdims=True)
        p = np.where(tot > 0, ex / np.where(tot > 0, tot, 1.0), 0.0)
        lse = (base + np.log(tot))[:, 0]
    return p, lse


def balance_loss(logits, idx, valid=None, offsets=None):
    """dict(loss [2], counts, mean_prob, lse, coef, norm)."""
    s, e = logits.shape
    k = idx.shape[1]
    live = np.ones(s, bool) if valid is None else np.asarray(valid) != 0
    offsets = np.array([0, s]) if offsets is None else np.asarray(offsets)
    B = len(offsets) - 1
    counts, P, coef = np.zeros((B, e), np.int64), np.zeros((B, e)), np.zeros((B, e))
    lse = np.zeros(s)
    loss, z, nseq, T = 0.0, 0.0, 0, 0
    for b in range(B):
        rows = np.arange(offsets[b], offsets[b + 1])
        rows = rows[live[rows]]
        if not len(rows):
            continue
        p, l = _softmax(logits[rows])
        lse[rows] = l
        for j in idx[rows].reshape(-1):
            if 0 <= j < e:
                counts[b, j] += 1
        n = len(rows)
        P[b] = p.sum(0) / n
        f = counts[b] / (k * n)
        coef[b] = e * f / n
        loss += e * float((f * P[b]).sum())
        z += float((l[~np.isneginf(l)] ** 2).sum())
        nseq, T = nseq + 1, T + n
    norm = np.array([1.0 / max(nseq, 1), 1.0 / max(T, 1)])
    return dict(loss=np.array([loss, z]) * norm, counts=counts, mean_prob=P, lse=lse, coef=coef, norm=norm)


def balance_loss_bwd(logits, lse, coef, norm, dloss, valid=None, offsets=None, add=None):
    s, e = logits.shape
    live = np.ones(s, bool) if valid is None else np.asarray(valid) != 0
    offsets = np.array([0, s]) if offsets is None else np.asarray(offsets)
    d = np.zeros((s, e)) if add is None else add.astype(np.float64).copy()
    for b in range(len(offsets) - 1):
        for t in range(offsets[b], offsets[b + 1]):
            if not live[t] or np.isneginf(lse[t]):
                continue
            p = np.exp(logits[t] - lse[t])
            d[t] += dloss[0] * norm[0] * p * (coef[b] - (coef[b] * p).sum()) + dloss[1] * norm[1] * 2 * lse[t] * p
    return d


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    assert kind == "silu"
    return z / (1.0 + np.exp(-z))


def act_slope(z, kind):
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    sg = 1.0 / (1.0 + np.exp(-z))
    return sg * (1.0 + z * (1.0 - sg))


def linear(x, W, b=None, kind="none", residual=None):
    """(y, z): z = x W^T + b, y = act(z) + residual."""
    z = x @ W.T
    if b is not None:
        z = z + b
    y = act(z, kind)
    if residual is not None:
        y = y + residual
    return y, z


def linear_bwd(dy, x, W, z=None, kind="none"):
    """(dx, dW, db, dz)."""
    dz = dy if kind == "none" else dy * act_slope(z, kind)
    return dz @ W, dz.T @ x, dz.sum(0), dz
