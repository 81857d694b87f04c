"""Oracle softmax cross entropy from hidden states and its gradients (float64).

Test infrastructure only; see ``oracle/__init__.py``. Per token with x = h W^T, z = x or c tanh(x / c),
lse = log sum_v exp(z_v), target y, label smoothing eps and z-loss lam:

    L       = (1 - eps) (lse - z_y) + eps (lse - mean_v z_v) + lam lse^2
    dL/dx_v = ((1 + 2 lam lse) p_v - (1 - eps) [v = y] - eps / V) (1 - (z_v / c)^2)
"""
from __future__ import annotations

import numpy as np


def row_loss(x, y, eps=0.0, lam=0.0, cap=0.0):
    """(loss, dL/dx, parts) of one row; NaN loss for a target outside the row."""
    x = np.asarray(x, np.float64)
    V = x.shape[0]
    z, d = x, np.ones(V)
    if cap:
        t = np.tanh(x / cap)
        z, d = cap * t, 1.0 / np.cosh(np.clip(x / cap, -300, 300)) ** 2
    m = np.max(z)
    e = np.exp(z - m)
    tot = np.sum(e)
    lse = m + np.log(tot)
    logp = (z - m) - np.log(tot)
    hot = np.zeros(V)
    if not 0 <= y < V:
        return np.nan, np.full(V, np.nan), dict(logp=logp, lse=lse, p=e / tot, z=z, d=d)
    hot[y] = 1.0
    loss = -(1.0 - eps) * logp[y] - eps * np.mean(logp) + lam * lse * lse
    dz = (1.0 + 2.0 * lam * lse) * (e / tot) - (1.0 - eps) * hot - eps / V
    return loss, dz * d, dict(logp=logp, lse=lse, p=e / tot, z=z, d=d)


def lmhead(h, W, target, mask, scale, w=None, eps=0.0, lam=0.0, cap=0.0):
    """Per-token loss, log p_y and lse, dx [T, V], d_h and dW of hidden states h and embedding W."""
    h, W = np.asarray(h, np.float64), np.asarray(W, np.float64)
    T, V = h.shape[0], W.shape[0]
    out = dict(loss=np.zeros(T), logp=np.zeros(T), lse=np.zeros(T), dx=np.zeros((T, V)), parts=[None] * T)
    hz = h.copy()
    for t in range(T):
        if mask is not None and not mask[t]:
            hz[t] = 0.0
            continue
        loss, dx, parts = row_loss(W @ h[t], int(target[t]), eps, lam, cap)
        out["loss"][t], out["lse"][t], out["parts"][t] = loss, parts["lse"], parts
        out["logp"][t] = parts["logp"][target[t]] if 0 <= target[t] < V else np.nan
        out["dx"][t] = dx * scale * (1.0 if w is None else float(w[t]))
    out["d_h"], out["dW"] = out["dx"] @ W, out["dx"].T @ hz
    return out


def clip(grads, max_norm, scale=1.0):
    """(norm, factor, each tensor's norm) of scaled gradients: factor = scale min(1, max_norm / norm)."""
    sums = np.array([np.sum(np.asarray(g, np.float64) ** 2) for g in grads])
    norm = scale * np.sqrt(np.sum(sums))
    if not np.isfinite(norm):
        return norm, 0.0, scale * np.sqrt(sums)
    return norm, scale * (max_norm / norm if norm > max_norm else 1.0), scale * np.sqrt(sums)
