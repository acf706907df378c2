"""Distillation of a drafter from the target's top alternatives (oracle; test infrastructure).

Plain float64 restatements of ssv_distill and its gradient, one row at a time
(include/ssv.h; the DFlash review, section 3.1, gives the position weight of a
draft loss, no interface).
"""
from __future__ import annotations

import numpy as np

RENORM, REST = 0, 1


def target(token: np.ndarray, value: np.ndarray, mode: int, V: int):
    """(dense p [V], listed [V], r): the target of a row; a token listed twice counts with both probabilities."""
    there = token >= 0
    t = np.asarray(value, np.float64)[there]
    p = np.zeros(V)
    listed = np.zeros(V, bool)
    listed[token[there]] = True
    if mode == REST:
        w = np.exp(t)
        r = max(0.0, 1.0 - w.sum())
    else:
        w = np.exp(t - t.max()) if len(t) and t.max() != -np.inf else np.zeros(len(t))
        w = w / w.sum() if w.sum() > 0 else w
        r = 0.0
    np.add.at(p, token[there], w)
    return p, listed, r


def row_distill(z: np.ndarray, token: np.ndarray, value: np.ndarray, T: float, mode: int, weight: float = 1.0):
    """(loss, gradient [V], stats [4]) of one row; the maximum is taken off first, so that rows far from 0 keep their digits."""
    z = np.asarray(z, np.float64)
    V = len(z)
    if weight == 0:
        return 0.0, np.zeros(V), np.zeros(4)
    p, listed, r = target(np.asarray(token), value, mode, V)
    if r < 2.0 ** -20 and not (z[~listed] >= z.max() - 100 * T).any():
        r = 0.0                                    # the drafter leaves the others nothing: a rounding of the list
    P = p.sum() + r
    if (z == -np.inf).all():
        return (weight * np.inf * P if P != 0 else 0.0), np.zeros(V), np.array([-np.inf, 0.0, -np.inf, 0.0])
    m = z.max()
    x = (z - m) / T
    S = np.exp(x).sum()
    logq = x - np.log(S)
    others = z[~listed]
    mo = others.max() if len(others) else -np.inf
    So = np.exp((others - mo) / T).sum() if mo > -np.inf else 0.0
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):   # share: of the others alone
        ln_u = (mo - m) / T + np.log(So) - np.log(S)
        loss = np.sum(np.where(p > 0, p * (np.log(np.where(p > 0, p, 1.0)) - logq), 0.0))
        if r > 0:
            loss += r * (np.log(r) - ln_u)
        share = np.exp((z - mo) / T) / So if So > 0 else np.zeros(V)   # of an other token among the others
        grad = np.where(listed, P * np.exp(logq) - p, share * (P * np.exp(ln_u) - r)) * (weight / T)
    return weight * loss, grad, np.array([m, S, mo, So])


def log_rest(stats: np.ndarray, T: float) -> float:
    """ln u from a row's statistics."""
    m, S, mo, So = stats
    return (mo - m) / T + np.log(So) - np.log(S) if So > 0 else -np.inf


def distill_batch(z, token, value, T, mode, weight=None):
    """(loss [n], grad [n, V], stats [n, 4])."""
    n = len(z)
    w = np.ones(n) if weight is None else weight
    rows = [row_distill(z[i], token[i], value[i], T, mode, float(w[i])) for i in range(n)]
    return (np.array([r[0] for r in rows]), np.stack([r[1] for r in rows]) if n else np.zeros(np.shape(z)),
            np.array([r[2] for r in rows]).reshape(n, 4))
