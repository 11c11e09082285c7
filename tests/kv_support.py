"""Inputs and calls shared by the GPU tests of the 4-bit cache."""

from __future__ import annotations

import numpy as np
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev
from oracle import kv_oracle as ko

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def desc_of(lay: ko.Layout, scale=0.0) -> svr.KvDesc:
    return svr.KvDesc(lay.heads, lay.kv_heads, lay.dim, lay.page, lay.window, lay.rotary,
                      lay.interleaved, scale, lay.eps)


class Plan:
    """Offsets, lengths and a shuffled page table of sequences with `rows` new rows and `lens` tokens."""

    def __init__(self, lay, rows, lens, rng, pad_rows=0, spare=2, width=None):
        self.lay = lay
        self.offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.lens = np.asarray(lens, dtype=np.int32)
        used = [min(max(0, -(-int(n) // lay.page)), width or 1 << 30) for n in lens]
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        w = width or max(max(used), 1)
        # Entries that no token needs point nowhere, at either side.
        self.table = np.where(rng.random((len(lens), w)) < 0.5, -1, self.n_pages + 5).astype(np.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.T = int(self.offsets[-1]) + pad_rows
        self.max_rows = max(max(rows), 1)

    def batch(self) -> svr.KvBatch:
        return svr.KvBatch(dev(self.offsets), dev(self.lens), dev(self.table), self.max_rows)

    def empty_cache(self, fill=0xFF) -> np.ndarray:
        return np.full((self.n_pages, self.lay.kv_heads, self.lay.page_bytes), fill, dtype=np.uint8)

    def filled_cache(self, rng) -> np.ndarray:
        """Random codes and scales of 2^-3..2^1 where tokens are, 0xFF (NaN) everywhere else."""
        lay, c = self.lay, self.empty_cache()
        for b, n in enumerate(self.lens):
            for t in range(int(n)):
                at = ko.slot(lay, self.table[b], self.n_pages, t)
                if at is None:
                    continue
                for h in range(lay.kv_heads):
                    kc, vc, ks, vs = ko.page_parts(lay, c[at[0], h])
                    kc[at[1]] = rng.integers(0, 256, lay.dim // 2)
                    vc[at[1]] = rng.integers(0, 256, lay.dim // 2)
                    ks[at[1]] = rng.integers(124, 127, lay.dim // 32)
                    vs[at[1]] = rng.integers(124, 129, lay.dim // 32)
        return c


def rounded(x: np.ndarray, dtype: str):
    """The array as a device tensor of the type, and the float64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TYPES[dtype])
    return t.cuda(), t.double().numpy()


def attention_tolerance(dtype, out, size, reach, seen, dim):
    """Bound of |out - exact|, element by element.

    Rounding of the result: eps/2 of it.  A softmax weight carries its own
    rounding w (bf16: one term, eps/2 = 2^-8; fp16: two terms of 8 bits,
    2^-16; fp32: three, 2^-24), that of its score, at most dim + 4 roundings
    of 2^-24 of sum |scale q k| (which enters the weight and, with the sum of
    weights below the fraction, twice), the exponential's and the rescalings'
    (a few 2^-24, one for each step over the tokens: taken as 64), and the
    roundings of the sums over the tokens, 2^-24 for each token, above and
    below the fraction.  All of these scale with sum weight |value|.
    """
    w = {"bf16": 2.0 ** -8, "f16": 2.0 ** -16, "f32": 2.0 ** -24}[dtype]
    u = 2.0 ** -24
    rel = w + 2 * (dim + 4) * u * reach[:, :, None] + (64 + 2 * seen[:, None, None]) * u
    # fp16 results below its normal range round to half of 2^-24.
    return torch.finfo(TYPES[dtype]).eps / 2 * np.abs(out) * (1 + rel) + rel * size + 2.0 ** -25
