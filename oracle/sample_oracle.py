"""CPU oracle of sampled verification (test infrastructure only).

Float64 NumPy, sequence by sequence and draft by draft, of what
``include/moe_sample.h`` documents, with every distribution normalised where it
changes.  Shares no code with the library.
"""

from __future__ import annotations

import numpy as np

from . import tree_oracle as to

LARGEST = float(np.finfo(np.float32).max)


def distribution(x, temperature):
    """The target's probabilities of one row of logits, or None where it has none."""
    x = np.asarray(x, np.float64).copy()
    x[np.isnan(x) | (x <= -LARGEST)] = -np.inf
    x[np.isposinf(x)] = LARGEST
    if np.isneginf(x).all():
        return None
    p = np.zeros_like(x)
    if not temperature >= 2.0 ** -126:
        p[np.argmax(x)] = 1.0
        return p
    some = x > -np.inf
    e = np.exp((x[some] - x.max()) / min(temperature, 2.0 ** 64))
    p[some] = e / e.sum()
    return p


def pick(p, u):
    """The first column whose cumulative weight is above u of the whole, and how far the nearest border lies."""
    cum = np.cumsum(p)
    above = np.flatnonzero((cum > u * cum[-1]) & (p > 0))
    col = int(above[0]) if len(above) else int(np.flatnonzero(p > 0)[-1])
    return col, float(np.min(np.abs(cum[p > 0] - u * cum[-1])) / cum[-1])


def sequence(logits, parents, tokens, draft_probs, temperature, accept_u, sample_u, off, rows, most):
    """Accepted rows from the root on, tokens, and the smallest distance from any border (of probability 1)."""
    V = logits.shape[1]
    path, out, margin = [0], [], np.inf
    while True:
        r = off + path[-1]
        p = distribution(logits[r], temperature)
        greedy = not temperature >= 2.0 ** -126
        best = None if p is None else int(np.argmax(p))  # (equal ones: the lower column)
        went = None
        for c in to.children(parents, off, rows, path[-1], most):
            t, u = int(tokens[off + c]), float(accept_u[off + c])
            if p is None or not 0 <= t < V:
                continue
            if greedy:
                if t == best:
                    went = c
                    break
                continue
            if draft_probs is None:
                limit = u
                after = p.copy()
                after[t] = 0.0
            else:
                q = np.asarray(draft_probs[r], np.float64)
                q = np.where(q > 0, q, 0.0)
                limit = u * q[t]
                after = np.maximum(p - q, 0.0)
            margin = min(margin, abs(limit - p[t]) if p[t] > 0 else np.inf)
            if limit < p[t]:
                went = c
                break
            # What is left of what was left: normalised again.
            p = after / after.sum() if after.sum() > 0 else after
        if went is None:
            if p is None:
                out.append(-1)
            elif p.sum() == 0 or greedy:
                out.append(best)
            else:
                t, far = pick(p, float(sample_u))
                margin = min(margin, far)
                out.append(t)
            return path, out, margin
        path.append(went)
        out.append(int(tokens[off + went]))


def verify(logits, offsets, parents, tokens, accept_u, sample_u, max_rows, max_children, draft_probs=None,
           temperature=None):
    """accepted and path [B][max_rows] (-1 behind), n_accepted [B], the sequences' last rows (of the
    batch) and the smallest distance of any decision from its border; None in the place of a sequence without rows."""
    res = dict(accepted=[], path=[], n_accepted=[], row=[], margin=np.inf)
    for b in range(len(offsets) - 1):
        off, rows = int(offsets[b]), min(int(offsets[b + 1] - offsets[b]), max_rows)
        if rows == 0:
            for k in ("accepted", "path", "n_accepted", "row"):
                res[k].append(None)
            continue
        t = 1.0 if temperature is None else float(temperature[b])
        path, out, margin = sequence(logits, parents, tokens, draft_probs, t, accept_u, sample_u[b], off, rows,
                                     max_children)
        res["margin"] = min(res["margin"], margin)
        res["accepted"].append(out + [-1] * (max_rows - len(out)))
        res["path"].append(path + [-1] * (max_rows - len(path)))
        res["n_accepted"].append(len(path) - 1)
        res["row"].append(off + path[-1])
    return res
