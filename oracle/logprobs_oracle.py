"""CPU oracle of log probabilities, entropy and top alternatives (test
infrastructure only): float64 NumPy of what ``include/moe_logprobs.h`` documents."""

from __future__ import annotations

import math

import numpy as np


def row_logprobs(row) -> np.ndarray:
    """Log probability of every column of one row."""
    x = np.asarray(row, dtype=np.float64)
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.full(x.shape, np.nan)
    m = x.max()
    if m == -np.inf:
        return np.full(x.shape, -np.inf)
    return x - m - math.log(math.fsum(np.exp(x - m)))


def entropy(row) -> float:
    lp = row_logprobs(row)
    if np.isnan(lp).any():
        return math.nan
    p = np.exp(lp)
    return -math.fsum((p * np.where(p > 0, lp, 0.0)).tolist())


def top_columns(row, k: int) -> list:
    """The k columns by value, equal ones by the lower column; NaN as -inf."""
    x = np.asarray(row, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    return sorted(range(len(x)), key=lambda c: (-x[c], c))[:k] if len(x) <= 4096 else \
        np.lexsort((np.arange(len(x)), -x))[:k].tolist()


def logprobs(logits, targets, k: int) -> dict:
    L = np.asarray(logits)
    lp = [row_logprobs(r) for r in L]
    ids = [top_columns(r, k) for r in L]
    return dict(
        logprobs=np.array([p[t] if 0 <= t < len(p) else np.nan for p, t in zip(lp, targets)]),
        entropy=np.array([entropy(r) for r in L]), top_ids=np.array(ids, dtype=np.int64).reshape(len(L), k),
        top_logprobs=np.array([p[i] for p, i in zip(lp, ids)]).reshape(len(L), k))
