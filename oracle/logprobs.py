"""Log-probabilities of a pass's logits (oracle; test infrastructure).

Plain float64 restatements of ssv_logprobs, one row at a time: log-probability
and rank of a token, entropy, log-sum-exp and top alternatives (include/ssv.h;
the pages have no interface for them).
"""
from __future__ import annotations

import numpy as np


def order(row: np.ndarray) -> np.ndarray:
    """Tokens by descending logit, equal ones by index; NaN left out."""
    idx = np.nonzero(~np.isnan(row))[0]
    return idx[np.lexsort((idx, -row[idx]))]


def row_logprobs(row: np.ndarray, token: int, top_k: int, T: float):
    """(logprob, rank, entropy, lse, top_logprob [top_k], top_token [top_k]) of one row; token -1: logprob and rank None."""
    row = np.asarray(row, np.float64)
    by = order(row)
    tops = by[row[by] > -np.inf][:top_k]
    top_token = np.full(top_k, -1, np.int64)
    top_token[:len(tops)] = tops
    top_logprob = np.full(top_k, -np.inf)
    rank = None if token < 0 else (0 if np.isnan(row[token]) else int(np.nonzero(by == token)[0][0]) + 1)
    if np.isnan(row).any() or (row == np.inf).any():
        top_logprob[:len(tops)] = np.nan
        return (None if token < 0 else np.nan), rank, np.nan, np.nan, top_logprob, top_token
    if (row == -np.inf).all():
        return (None if token < 0 else -np.inf), rank, 0.0, -np.inf, top_logprob, top_token
    m = row.max()
    x = (row - m) / T
    e = np.exp(x)
    S = e.sum()
    lp = x - np.log(S)
    entropy = -np.sum(np.where(e > 0, e / S * np.where(e > 0, lp, 0.0), 0.0))
    top_logprob[:len(tops)] = lp[tops]
    return (None if token < 0 else lp[token]), rank, entropy, m / T + np.log(S), top_logprob, top_token


def logprobs_batch(logits: np.ndarray, tokens, rows, top_k: int, T: float):
    """ssv_logprobs of every entry, as arrays; idle entries (token or row -1) give 0, -1 and -inf."""
    n = len(tokens) if tokens is not None else len(rows) if rows is not None else len(logits)
    out = dict(logprob=np.zeros(n), rank=np.zeros(n, np.int64), entropy=np.zeros(n), lse=np.zeros(n),
               top_logprob=np.full((n, top_k), -np.inf), top_token=np.full((n, top_k), -1, np.int64))
    for i in range(n):
        r = i if rows is None else int(rows[i])
        t = -2 if tokens is None else int(tokens[i])
        if r == -1 or t == -1:
            continue
        lp, rank, ent, lse, tl, tt = row_logprobs(logits[r], t, top_k, T)
        if tokens is not None:
            out["logprob"][i], out["rank"][i] = lp, rank
        out["entropy"][i], out["lse"][i], out["top_logprob"][i], out["top_token"][i] = ent, lse, tl, tt
    return out
