"""Oracle distillation loss over a teacher's top tokens and its gradient (float64).

Test infrastructure only; see ``oracle/__init__.py``. For a student row z, a temperature tau and the
teacher's list of (token, log-prob) entries (token -1: unused), with p = softmax(z/tau), S the listed
tokens, Q = sum_S q, q_R = 1 - Q and p_R = sum of p outside S:

    FORWARD_TOPK  L = sum_S (q/Q) log((q/Q) / p)
    FORWARD_TAIL  L = sum_S q log(q/p) + q_R log(q_R/p_R)
    REVERSE_TAIL  L = sum_S p log(p/q) + p_R log(p_R/q_R)

with 0 log 0 = 0, no remainder term where S is the whole row or empty (loss and gradient 0), and a q_R
below 2^-24 counted as 0 (FORWARD_TAIL; below 2^-16 where every token outside S is 2^126 times less probable than
the row's most probable) or as 2^-24 (REVERSE_TAIL). The gradient is dL/dz.
"""
from __future__ import annotations

import numpy as np

from .loss import as_f64
from .score import range_limit

FORWARD_TOPK, FORWARD_TAIL, REVERSE_TAIL = 0, 1, 2
TAIL_MIN = 2.0 ** -24
TAIL_NONE = 2.0 ** -16


def row_loss(z, idx, tlogp, kind, tau=1.0):
    """(loss, dL/dz, parts) of one row; NaN throughout for a bad list or row."""
    z = as_f64(np.asarray(z))
    V = z.shape[0]
    idx, tlogp = np.asarray(idx), np.asarray(tlogp, np.float64)
    on = idx != -1
    S, lq = idx[on], tlogp[on]
    bad = (np.any(S < 0) or np.any(S >= V) or len(set(S.tolist())) != len(S) or np.any(np.isnan(lq))
           or np.any(lq == np.inf))
    with np.errstate(invalid="ignore"):
        z = np.where(z < -range_limit(tau), -np.inf, z)
    m = np.max(z)
    if bad or not np.isfinite(m) or m > range_limit(tau):
        return np.nan, np.full(V, np.nan), None
    d = (z - m) / float(tau)
    e = np.exp(d)
    tot = np.sum(e)
    p, lp = e / tot, d - np.log(tot)
    out = np.ones(V, bool)
    out[S] = False
    # the mass outside the list, by its logarithm: as a share of the row it may underflow
    mo = np.max(d[out]) if out.any() else -np.inf
    w = np.exp(d[out] - mo) if mo > -np.inf else np.zeros(int(out.sum()))
    lr = mo + np.log(np.sum(w)) - np.log(tot) if mo > -np.inf else -np.inf
    pr = float(np.exp(lr))
    q = np.exp(lq)
    dx = np.zeros(V)
    parts = dict(p=p, lp=lp, pr=pr, m=m, tot=tot, out=out)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if kind == FORWARD_TOPK:
            if not len(S) or not np.any(lq > -np.inf):
                return 0.0, dx, dict(parts, q=np.zeros(len(S)), alpha=0.0)
            mx = np.max(lq)
            q = np.exp(lq - mx)
            lq = lq - mx - np.log(q.sum())
            q = q / q.sum()
            loss = float(np.sum(np.where(q > 0, q * (lq - lp[S]), 0.0)))
            dx = p.copy()
            dx[S] -= q
            return loss, dx / tau, dict(parts, q=q, alpha=1.0)
        if not len(S):  # no list: nothing to learn (1 log(1/1), the gradient of a constant)
            return 0.0, dx, dict(parts, q=q, qr=0.0, alpha=0.0, f=q, fr=0.0)
        qr = 1.0 - q.sum()
        if kind == FORWARD_TAIL:
            qr = 0.0 if qr < (TAIL_MIN if mo >= -126 * np.log(2) else TAIL_NONE) or not out.any() else qr
            loss = float(np.sum(np.where(q > 0, q * (lq - lp[S]), 0.0)))
            loss += qr * (np.log(qr) - lr) if qr > 0 else 0.0
            mass = q.sum() + qr  # d/dx of -sum q_i log p_i is (sum q) p - q
            alpha = mass - (qr / np.float64(pr) if qr > 0 else 0.0)
            dx[out] = mass * p[out] - (qr * w / np.sum(w) if qr > 0 else 0.0)
            dx[S] = mass * p[S] - q
            return loss, dx / tau, dict(parts, q=q, qr=qr, alpha=alpha)
        qr = max(qr, TAIL_MIN)
        tail = pr > 0
        f = np.where(p[S] > 0, lp[S] - lq, 0.0)
        fr = lr - np.log(qr) if tail else 0.0
        loss = float(np.sum(p[S] * f) + pr * fr)
        dx[out] = p[out] * (fr - loss)
        dx[S] = p[S] * (f - loss)
        dx[p == 0] = 0.0
        return loss, dx / tau, dict(parts, q=q, qr=qr, f=f, fr=fr, alpha=fr - loss if tail else 0.0)
