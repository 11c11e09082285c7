"""CPU oracle of a verify step on trees of drafts (test infrastructure only).

Plain NumPy, row by row, of what ``include/moe_tree.h`` documents: which rows of
a tree see which, attention over the stored values with that, and the move of an
accepted path's bytes.  Shares no code with the library.
"""

from __future__ import annotations

import numpy as np

from . import kv_oracle as ko


def parent(parents, off, i):
    """The parent's place of row i of a sequence that begins at `off`, or -1."""
    if i == 0:
        return -1
    p = i - 1 if parents is None else int(parents[off + i])
    return p if 0 <= p < i else -1


def children(parents, off, rows, i, most):
    return [j for j in range(i + 1, rows) if parent(parents, off, j) == i][:most]


def ancestors(parents, off, i):
    """Row i and those it hangs on, from the root on."""
    out = [i]
    while (p := parent(parents, off, out[0])) >= 0:
        out.insert(0, p)
    return out


def plan(offsets, parents, lens, max_rows, words):
    """mask uint64 [T][words], positions int64 [T], and which rows have them."""
    T = int(offsets[-1])
    mask, pos, on = np.zeros((T, words), np.uint64), np.zeros(T, np.int64), np.zeros(T, bool)
    for b in range(len(offsets) - 1):
        off, rows = int(offsets[b]), int(offsets[b + 1] - offsets[b])
        for i in range(min(rows, max_rows)):
            seen = ancestors(parents, off, i)
            for j in seen:
                mask[off + i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
            pos[off + i] = int(lens[b]) - rows + len(seen) - 1
            on[off + i] = True
    return mask, pos, on


def attention(lay: ko.Layout, cache, offsets, lens, table, q, mask, max_rows, scale=None):
    """As kv_oracle.attention, for rows that see the new rows marked in mask uint64 [T][words]."""
    T, words = q.shape[0], mask.shape[1]
    scale = 1.0 / np.sqrt(lay.dim) if scale is None else scale
    out, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, reach = np.full(q.shape[:2], np.nan), np.full(q.shape[:2], np.nan)
    seen_n = np.zeros(T, int)
    G = lay.heads // lay.kv_heads
    for b in range(len(lens)):
        rows = int(offsets[b + 1] - offsets[b])
        base = int(lens[b]) - rows
        n = max(int(min(lens[b], len(table[b]) * lay.page)), 0)
        rows = min(rows, max_rows)
        for h in range(lay.kv_heads):
            if rows == 0:
                continue
            K, V, there = ko.stored(lay, cache, table[b], n, h)
            for m in range(rows):
                i = int(offsets[b]) + m
                places = list(range(max(base, 0)))
                for j in range(min(rows, 64 * words)):
                    if int(mask[i, j // 64]) >> (j % 64) & 1:
                        places.append(base + j)
                if lay.window:
                    places = places[-lay.window:]
                places = [p for p in places if 0 <= p < n and there[p]]
                seen_n[i] = len(places)
                for hh in range(h * G, (h + 1) * G):
                    if not places:
                        out[i, hh], size[i, hh], lse[i, hh], reach[i, hh] = 0, 0, -np.inf, 0
                        continue
                    qv = np.asarray(q[i, hh], np.float64)
                    s = K[places] @ qv * scale
                    reach[i, hh] = np.max(np.abs(K[places]) @ np.abs(qv)) * scale
                    m0 = np.max(s)
                    w = np.exp(s - m0)
                    out[i, hh] = w @ V[places] / w.sum()
                    size[i, hh] = w @ np.abs(V[places]) / w.sum()
                    lse[i, hh] = m0 + np.log(w.sum())
    return out, lse, size, reach, seen_n


def commit(lay: ko.Layout, cache, offsets, lens, table, max_rows, path, n_accepted):
    """Moves the paths' bytes in `cache` (uint8 [pages][kv heads][page bytes]); returns the kept lengths."""
    old = cache.copy()
    kept = []
    for b in range(len(lens)):
        rows = int(offsets[b + 1] - offsets[b])
        base = int(lens[b]) - rows
        n = max(min(int(n_accepted[b]), min(rows, max_rows) - 1, path.shape[1] - 1), 0)
        kept.append(base + n + 1 if rows else int(lens[b]))
        for i in range(1, n + 1):
            r = int(path[b, i])
            if not i < r < min(rows, max_rows):
                continue
            src, dst = (ko.slot(lay, table[b], len(cache), base + x) for x in (r, i))
            if src is None or dst is None:
                continue
            for h in range(lay.kv_heads):
                for new, was in zip(ko.page_parts(lay, cache[dst[0], h]), ko.page_parts(lay, old[src[0], h])):
                    new[dst[1]] = was[src[1]]
    return np.array(kept)
