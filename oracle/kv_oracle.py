"""CPU oracle of the paged 4-bit key/value cache (test infrastructure only).

Plain float64 NumPy, token by token, of what ``include/moe_kv.h`` documents:
head norms, position rotation, 4-bit blocks, the byte layout of a page, and
attention over the stored values.  Shares no code with the library.
"""

from __future__ import annotations

import dataclasses

import numpy as np

# The magnitudes of codes 0..7; bit 3 is the sign.
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@dataclasses.dataclass
class Layout:
    heads: int
    kv_heads: int
    dim: int
    page: int = 64
    window: int = 0
    rotary: int = 0
    interleaved: bool = False
    eps: float = 1e-6

    @property
    def page_bytes(self) -> int:
        return self.page * (self.dim + self.dim // 16)


def block_codes(x):
    """Codes [32] and scale byte of one block of 32 finite values."""
    x = np.asarray(x, dtype=np.float64)
    top = np.max(np.abs(x))
    e = 0
    if top > 0:
        e = -126
        while e < 125 and top > 7.0 * 2.0 ** e:
            e += 1
    codes = np.zeros(32, dtype=np.uint8)
    for i, v in enumerate(x):
        t = abs(v) / 2.0 ** e
        off = np.abs(MAGNITUDES - t)
        near = np.flatnonzero(off == off.min())
        code = near[0] if len(near) == 1 else next(c for c in near if c % 2 == 0)
        codes[i] = code | (8 if v < 0 else 0)
    return codes, e + 127


def vector_bytes(x):
    """Code bytes [D/2] and scale bytes [D/32] of one head vector."""
    blocks = [block_codes(b) for b in np.asarray(x).reshape(-1, 32)]
    c = np.concatenate([b[0] for b in blocks])
    return c[0::2] | c[1::2] << 4, np.array([b[1] for b in blocks], dtype=np.uint8)


def vector_values(code_bytes, scale_bytes):
    """The float64 values of one head vector (NaN under scale byte 255)."""
    c = np.empty(2 * len(code_bytes), dtype=np.int64)
    c[0::2], c[1::2] = code_bytes & 15, code_bytes >> 4
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scale_bytes == 255, np.nan, 2.0 ** (scale_bytes.astype(np.float64) - 127))
    return v * np.repeat(s, 32)


def page_parts(lay: Layout, page):
    """Views of one head's page: code bytes of keys, of values, scale bytes of keys, of values."""
    P, D = lay.page, lay.dim
    a, b = P * D // 2, P * D // 32
    return (page[:a].reshape(P, D // 2), page[a:2 * a].reshape(P, D // 2),
            page[2 * a:2 * a + b].reshape(P, D // 32), page[2 * a + b:].reshape(P, D // 32))


def head_vector(lay: Layout, x, w, inv_freq, pos):
    """One head's normed and rotated vector, float64."""
    y = np.asarray(x, dtype=np.float64).copy()
    if w is not None:
        y = y / np.sqrt(np.mean(y * y) + np.float64(np.float32(lay.eps))) * np.asarray(w, np.float64)
    R = lay.rotary
    for j in range(R // 2):
        a, b = (2 * j, 2 * j + 1) if lay.interleaved else (j, j + R // 2)
        t = float(pos) * float(inv_freq[j])
        y[a], y[b] = y[a] * np.cos(t) - y[b] * np.sin(t), y[b] * np.cos(t) + y[a] * np.sin(t)
    return y


def slot(lay: Layout, table_row, n_pages, place):
    """(page, token of the page) of a place, or None where there is none."""
    if place < 0 or place // lay.page >= len(table_row):
        return None
    page = int(table_row[place // lay.page])
    return (page, place % lay.page) if 0 <= page < n_pages else None


def append(lay: Layout, cache, offsets, lens, table, q, k, v, q_norm=None, k_norm=None,
           inv_freq=None, positions=None):
    """Writes the rows into `cache` (uint8 [pages][kv heads][page bytes]); returns q_out float64
    (NaN in rows of no sequence)."""
    q_out = np.full(q.shape, np.nan)
    for b in range(len(lens)):
        for i in range(offsets[b], offsets[b + 1]):
            place = int(lens[b]) - int(offsets[b + 1]) + i
            pos = place if positions is None else positions[i]
            for h in range(lay.heads):
                q_out[i, h] = head_vector(lay, q[i, h], q_norm, inv_freq, pos)
            at = slot(lay, table[b], len(cache), place)
            if at is None:
                continue
            for h in range(lay.kv_heads):
                with np.errstate(all="ignore"):
                    key = head_vector(lay, k[i, h], k_norm, inv_freq, pos)
                val = np.asarray(v[i, h], np.float64)
                kc, vc, ks, vs = page_parts(lay, cache[at[0], h])
                if np.isfinite(key).all() and np.isfinite(val).all():
                    (kc[at[1]], ks[at[1]]), (vc[at[1]], vs[at[1]]) = vector_bytes(key), vector_bytes(val)
                else:
                    kc[at[1]], vc[at[1]], ks[at[1]], vs[at[1]] = 0, 0, 255, 127
    return q_out


def stored(lay: Layout, cache, table_row, n, h):
    """Keys and values [n][D] of places 0..n-1 and whether each is there."""
    K, V, there = np.zeros((n, lay.dim)), np.zeros((n, lay.dim)), np.zeros(n, bool)
    for t in range(n):
        at = slot(lay, table_row, len(cache), t)
        if at is not None:
            kc, vc, ks, vs = page_parts(lay, cache[at[0], h])
            K[t], V[t], there[t] = vector_values(kc[at[1]], ks[at[1]]), vector_values(vc[at[1]], vs[at[1]]), True
    return K, V, there


def attention(lay: Layout, cache, offsets, lens, table, q, scale=None):
    """out, lse, and for tolerances: sum of weight x |value|, largest sum of |scale q k| of a row,
    and the tokens seen (float64; rows of no sequence are NaN)."""
    T = q.shape[0]
    scale = 1.0 / np.sqrt(lay.dim) if scale is None else scale
    out, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, reach = np.full(q.shape[:2], np.nan), np.full(q.shape[:2], np.nan)
    seen_n = np.zeros(T, int)
    G = lay.heads // lay.kv_heads
    for b in range(len(lens)):
        rows = int(offsets[b + 1] - offsets[b])
        n = int(min(lens[b], len(table[b]) * lay.page))
        for h in range(lay.kv_heads):
            if rows == 0:
                continue
            K, V, there = stored(lay, cache, table[b], max(n, 0), h)
            for m in range(rows):
                i, place = offsets[b] + m, int(lens[b]) - rows + m
                t = np.arange(max(n, 0))
                see = there & (t <= place)
                if lay.window:
                    see &= t > place - lay.window
                seen_n[i] = see.sum()
                for hh in range(h * G, (h + 1) * G):
                    if not see.any():
                        out[i, hh], size[i, hh], lse[i, hh], reach[i, hh] = 0, 0, -np.inf, 0
                        continue
                    qv = np.asarray(q[i, hh], np.float64)
                    s = K[see] @ qv * scale
                    reach[i, hh] = np.max(np.abs(K[see]) @ np.abs(qv)) * scale
                    m0 = np.max(s)
                    w = np.exp(s - m0)
                    out[i, hh] = w @ V[see] / w.sum()
                    size[i, hh] = w @ np.abs(V[see]) / w.sum()
                    lse[i, hh] = m0 + np.log(w.sum())
    return out, lse, size, reach, seen_n
