"""Oracle token scoring (float64): log-probs, entropy and the top alternatives of a logits row.

Test infrastructure only; see ``oracle/__init__.py``. For a row of logits z and a temperature tau,

    log p_v = z_v/tau - log sum_u exp(z_u/tau),    H = -sum_v p_v log p_v   (0 log 0 = 0)

and the alternatives are the K largest logits in descending order, equal ones by ascending index.
A row with a NaN or +inf logit, or none above -inf, has no distribution: NaN and index -1. A logit
whose z log2(e)/tau lies below the float32 range (a mask by the type's lowest value; range_limit) has no
mass, as -inf has none; the order still goes by its value. One above the range counts as +inf.
"""
from __future__ import annotations

import numpy as np

from .loss import as_f64


def range_limit(tau):
    """The largest |z| within the float32 range after the scaling: by the power of two above the float32
    log2(e)/tau, the scale of logits past 2^31."""
    c = float(np.float32(np.log2(np.e) / float(tau)))
    return float(np.finfo(np.float32).max) / 2.0 ** (np.floor(np.log2(c)) + 1)


def score_row(z, y, K, tau=1.0):
    """(log p_y or NaN for a target outside the row, H, top indices, their log-probs)."""
    z = as_f64(np.asarray(z))
    V = z.shape[0]
    order = -z
    with np.errstate(invalid="ignore"):
        z = np.where(z < -range_limit(tau), -np.inf, z)
    m = np.max(z)
    if not np.isfinite(m) or m > range_limit(tau):
        return np.nan, np.nan, np.full(K, -1, np.int64), np.full(K, np.nan)
    d = (z - m) / float(tau)
    e = np.exp(d)
    lse = np.log(np.sum(e))
    with np.errstate(invalid="ignore"):
        H = lse - float(np.sum(np.where(e > 0, e * d, 0.0)) / np.sum(e))
    idx = np.argsort(order, kind="stable")[:K]
    logp = d[y] - lse if y is not None and 0 <= y < V else np.nan
    return float(logp), float(H), idx, d[idx] - lse
