"""One tree of so many rows that its row tiles fill the GPU (include/moe_tree.h): parts that run in
several rounds, row tiles that are not cut, and the workspace that a call asks for.

The oracle (oracle/tree_oracle.py) takes rows and heads one by one, too slow for these sizes: the
reference here is the same sums in float64 over all rows of a key/value head at once, compared with the
oracle at a small size first."""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev, log
from kv_support import TYPES, attention_tolerance, desc_of, rounded
from oracle import kv_oracle as ko, tree_oracle as to
from test_gpu_tree import TreePlan
from tree_support import as_words

pytestmark = pytest.mark.gpu


def reference(lay, plan, cache, q64):
    """What tree_oracle.attention gives for one sequence whose pages are all there."""
    rows, n = plan.max_rows, int(plan.lens[0])
    base, G = n - rows, lay.heads // lay.kv_heads
    bits = np.unpackbits(plan.mask[:rows].view(np.uint8), axis=1, bitorder="little")[:, :rows].astype(bool)
    seen = np.concatenate([np.ones((rows, base), bool), bits], 1)
    if lay.window:  # the last ones of what a row sees
        seen &= np.cumsum(seen[:, ::-1], 1)[:, ::-1] <= lay.window
    hidden = dev(~seen)
    out, size = (torch.empty((rows, lay.heads, lay.dim), dtype=torch.float64, device="cuda") for _ in range(2))
    lse, reach = (torch.empty((rows, lay.heads), dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(lay.kv_heads):
        K, V, there = ko.stored(lay, cache, plan.table[0], n, h)
        assert np.all(there)
        K, V = dev(K), dev(V)
        for hh in range(h * G, (h + 1) * G):
            q = dev(q64[:, hh])
            s = (q @ K.T) / np.sqrt(lay.dim)
            reach[:, hh] = ((q.abs() @ K.abs().T) / np.sqrt(lay.dim)).masked_fill(hidden, 0).amax(1)
            s = s.masked_fill(hidden, float("-inf"))
            lse[:, hh] = torch.logsumexp(s, 1)
            w = torch.softmax(s, 1)
            out[:, hh], size[:, hh] = w @ V, w @ V.abs()
    return [x.cpu().numpy() for x in (out, lse, size, reach)] + [seen.sum(1)]


def check_one(lay, rows, length, dtype, rng, kids=4, width=None):
    plan = TreePlan(lay, [rows], [length], rng, kids=kids, width=width)
    cache = plan.filled_cache(rng)
    q, q64 = rounded(rng.standard_normal((rows, lay.heads, lay.dim)), dtype)
    desc, batch, mask, c = desc_of(lay), plan.batch(), as_words(plan.mask), dev(cache)
    ws = svr.kv_workspace(desc, batch, rows)
    out, lse = torch.full_like(q, 77.0), torch.full((rows, lay.heads), 77.0, device="cuda")
    svr.moe_kv_tree_attention(desc, batch, mask, q, c, out, lse, ws=ws)
    again = torch.full_like(q, 77.0)
    svr.moe_kv_tree_attention(desc, batch, mask, q, c, again, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    want, rl, size, reach, seen = reference(lay, plan, cache, q64)
    tol = attention_tolerance(dtype, want, size, reach, seen, lay.dim)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= tol), (np.nanmax(err - tol), np.nanmax(err))
    # The score's roundings, the weights' sum (a rounding for each token), the logarithm and its sum.
    u = 2.0 ** -24
    t = (lay.dim + 4) * u * reach + (64 + seen[:, None]) * u + 8 * u * np.abs(rl)
    assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= t)


@pytest.mark.parametrize("window", [0, 21])
def test_the_reference_is_the_oracle(window):
    rng = np.random.default_rng(80)
    lay = ko.Layout(4, 2, 64, 16, window)
    plan = TreePlan(lay, [70], [150], rng, kids=3)
    cache = plan.filled_cache(rng)
    q64 = rng.standard_normal((70, 4, 64))
    a = reference(lay, plan, cache, q64)
    b = to.attention(lay, cache, plan.offsets, plan.lens, plan.table, q64, plan.mask, plan.max_rows)
    for x, y in zip(a, b):
        assert np.max(np.abs(x - y)) <= 1e-12 * max(1.0, np.max(np.abs(y)))


# (heads, KV heads, head size, type, rows, tokens, row tiles of a head that run at once: 256 compute units
# take two workgroups of these head sizes, three of 64 in fp16)
FULL = [
    (128, 8, 192, "f16", 70, 5200, 64), (128, 8, 192, "f16", 96, 2000, 64), (128, 8, 256, "bf16", 66, 5200, 64),
    (128, 8, 192, "f32", 80, 1500, 64), (64, 1, 64, "f32", 300, 5200, 512), (128, 8, 192, "bf16", 130, 5200, 64),
]
# Fewer row tiles than run at once, more parts.
CUT = [(64, 1, 64, "f16", 130, 8000, 768), (64, 1, 64, "f16", 96, 20000, 768)]


def row_tiles(heads, kv_heads, dim, dtype, rows):
    wide = {64: 32, 128: 32, 192: 32 if dtype == "bf16" else 16, 256: 16}[dim]
    return -(-rows * (heads // kv_heads) // wide)


@pytest.mark.parametrize("heads,kv_heads,dim,dtype,rows,length,at_once", FULL + CUT)
def test_one_tree_that_fills_the_gpu(heads, kv_heads, dim, dtype, rows, length, at_once):
    log(f"full {heads}/{kv_heads} D={dim} {dtype} {rows} rows, {length} tokens")
    case = (heads, kv_heads, dim, dtype, rows, length, at_once)
    assert (row_tiles(heads, kv_heads, dim, dtype, rows) > at_once) == (case in FULL)
    check_one(ko.Layout(heads, kv_heads, dim, 64), rows, length, dtype, np.random.default_rng(rows + dim))


@pytest.mark.parametrize("heads,kv_heads,dim,dtype,rows,length", [c[:6] for c in FULL + CUT] + [
    (64, 4, 192, "bf16", 61, 4000), (16, 1, 192, "bf16", 4, 9000), (64, 4, 192, "bf16", 7, 777)])
def test_a_workspace_is_asked_for_where_parts_use_it(heads, kv_heads, dim, dtype, rows, length):
    """A call that refuses a workspace of counters alone writes parts behind them, and no other call does."""
    log(f"workspace {heads}/{kv_heads} D={dim} {dtype} {rows} rows, {length} tokens")
    rng = np.random.default_rng(81)
    lay = ko.Layout(heads, kv_heads, dim, 64)
    plan = TreePlan(lay, [rows], [length], rng, kids=4)
    desc, batch, mask = desc_of(lay), plan.batch(), as_words(plan.mask)
    cache = torch.zeros((plan.n_pages, kv_heads, lay.page_bytes), dtype=torch.uint8, device="cuda")
    q = torch.ones((rows, heads, dim), dtype=TYPES[dtype], device="cuda")
    out = torch.empty_like(q)
    ws = svr.kv_workspace(desc, batch, rows)
    ws[svr._binding.KV_COUNTER_BYTES:] = 0xA5
    svr.moe_kv_tree_attention(desc, batch, mask, q, cache, out, ws=ws)
    used = bool((ws[svr._binding.KV_COUNTER_BYTES:] != 0xA5).any())
    try:
        svr.moe_kv_tree_attention(desc, batch, mask, q, cache, out, ws=ws[:svr._binding.KV_COUNTER_BYTES])
        refused = False
    except svr.MoeError as e:
        assert e.status == 4, e
        refused = True
    assert used == refused


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 40, 900])
@pytest.mark.parametrize("kids", [1, 3])
def test_the_largest_tree(dtype, window, kids):
    """1024 rows, masks of sixteen words; a chain, whose windows lie among the rows alone, and a tree."""
    log(f"1024 rows {dtype} W={window} kids={kids}")
    check_one(ko.Layout(4, 2, 64, 32, window), 1024, 1500, dtype, np.random.default_rng(82 + window), kids=kids)


# A table of 60000 tokens for fewer; row tiles of a head that run at once.
WIDE = [(64, 4, 192, "bf16", 65, 700, 128), (64, 4, 192, "bf16", 65, 2000, 128), (64, 4, 192, "bf16", 65, 20000, 128),
        (32, 8, 128, "bf16", 300, 700, 64), (128, 8, 192, "f16", 65, 2000, 64)]


@pytest.mark.parametrize("heads,kv_heads,dim,dtype,rows,length,at_once", WIDE)
def test_one_tree_that_is_short_for_its_table(heads, kv_heads, dim, dtype, rows, length, at_once):
    """Parts of twelve steps of four waves at least, or about as many as run at once (the last one of each row
    tile may be a short one more); what is written to the workspace says how many there are."""
    log(f"short {heads}/{kv_heads} D={dim} {dtype} {rows} rows, {length} tokens")
    lay = ko.Layout(heads, kv_heads, dim, 64)
    rng = np.random.default_rng(85 + length)
    check_one(lay, rows, length, dtype, rng, width=938)
    plan = TreePlan(lay, [rows], [length], rng, width=938)
    desc, batch = desc_of(lay), plan.batch()
    ws = svr.kv_workspace(desc, batch, rows)
    ws[svr._binding.KV_COUNTER_BYTES:] = 0xA5
    q = torch.ones((rows, heads, dim), dtype=TYPES[dtype], device="cuda")
    cache = torch.zeros((plan.n_pages, kv_heads, lay.page_bytes), dtype=torch.uint8, device="cuda")
    svr.moe_kv_tree_attention(desc, batch, as_words(plan.mask), q, cache, torch.empty_like(q), ws=ws)
    written = int((ws[svr._binding.KV_COUNTER_BYTES:].view(torch.int32) == 0).sum())  # sums of zeros
    n = row_tiles(heads, kv_heads, dim, dtype, rows)
    parts = written / (rows * heads * dim) * n  # of a head
    if length <= 2000:
        assert parts <= at_once + n
    else:
        assert parts > 2 * at_once
