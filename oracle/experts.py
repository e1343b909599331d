"""Plain 64-bit NumPy forms of the gated products, the experts' products over
row segments with their gradients, and gradient clipping.  Test
infrastructure only; shares nothing with the CUDA code.  Inputs are float64
arrays (the exact values of the bf16 or fp32 inputs)."""
from __future__ import annotations

import numpy as np

from .block import act, act_slope


def gated(x, W, b=None, kind="silu"):
    """(h, z): z = x W^T + b = [g | u], h = act(g) u."""
    z = x @ W.T
    if b is not None:
        z = z + b
    N = W.shape[0] // 2
    return act(z[:, :N], kind) * z[:, N:], z


def gated_dz(dh, z, kind="silu"):
    N = dh.shape[1]
    g, u = z[:, :N], z[:, N:]
    return np.concatenate([dh * u * act_slope(g, kind), dh * act(g, kind)], 1)


def gated_bwd(dh, x, W, z, kind="silu"):
    """(dx, dW, db, dz)."""
    dz = gated_dz(dh, z, kind)
    return dz @ W, dz.T @ x, dz.sum(0), dz


def segments(offsets, counts):
    """The rows of each expert, as slices."""
    return [slice(int(o), int(o) + int(n)) for o, n in zip(offsets, counts)]


def grouped_gated(X, W, segs, kind="silu"):
    """(H, Z); rows of no segment are NaN."""
    N = W.shape[1] // 2
    H, Z = np.full((X.shape[0], N), np.nan), np.full((X.shape[0], 2 * N), np.nan)
    for x, r in enumerate(segs):
        H[r], Z[r] = gated(X[r], W[x], None, kind)
    return H, Z


def grouped_bwd(dY, X, W, segs):
    """(dX, dW) of Y[r] = X[r] W[x]^T; rows of dX of no segment are NaN."""
    dX, dW = np.full(X.shape, np.nan), np.zeros(W.shape)
    for x, r in enumerate(segs):
        dX[r] = dY[r] @ W[x]
        dW[x] = dY[r].T @ X[r]
    return dX, dW


def clip(grads, max_norm):
    """(norm, coefficient)."""
    norm = np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))
