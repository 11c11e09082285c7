"""Trees of drafts and calls shared by the tests of the verify step on trees."""

from __future__ import annotations

import numpy as np
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev


def random_parents(rows, kids, rng, level_order=True):
    """Parents of a random tree: every row follows an earlier one that has room."""
    room, parent = [kids], [-1]
    for j in range(1, rows):
        open_ = [i for i in range(j) if room[i] > 0]
        p = open_[max(rng.integers(len(open_)), rng.integers(len(open_)))]
        room[p] -= 1
        room.append(kids)
        parent.append(p)
    if not level_order:
        return parent
    depth = [0] * rows
    for j in range(1, rows):
        depth[j] = depth[parent[j]] + 1
    order = sorted(range(rows), key=lambda j: (depth[j], j))
    new = {j: i for i, j in enumerate(order)}
    return [-1] + [new[parent[j]] for j in order[1:]]


def forest(row_counts, kids, rng, level_order=True):
    """offsets and parents (int32) of one tree a sequence."""
    offsets = np.concatenate([[0], np.cumsum(row_counts)]).astype(np.int32)
    parents = [p for n in row_counts if n for p in random_parents(n, kids, rng, level_order)]
    return offsets, np.array(parents, dtype=np.int32)


def tree_of(offsets, parents, max_rows, kids, pad_rows=0) -> svr.DraftTree:
    if parents is not None:
        parents = dev(np.concatenate([parents, np.full(pad_rows, -5)]).astype(np.int32))
    return svr.DraftTree(dev(np.asarray(offsets, np.int32)), parents, max_rows, kids)


def as_words(mask: np.ndarray) -> torch.Tensor:
    return dev(mask.view(np.int64))
