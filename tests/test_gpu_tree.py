"""Trees of drafts (include/moe_tree.h) on the GPU against the oracle (oracle/tree_oracle.py), every call
through the C ABI: masks and positions and the moved bytes have to be equal; attention within the bounds
that its causal form has (kv_support.attention_tolerance), since masks change which tokens are summed and
nothing else."""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev, log
from kv_support import TYPES, Plan, attention_tolerance, desc_of, rounded
from oracle import kv_oracle as ko, tree_oracle as to
from tree_support import as_words, forest, random_parents, tree_of

pytestmark = pytest.mark.gpu


# ---- plan

def check_plan(offsets, parents, lens, max_rows, words=None, pad=2):
    tree = tree_of(offsets, parents, max_rows, 1024, pad)
    words = words or tree.mask_words
    T = int(offsets[-1])
    mask = torch.full((T + pad, words), 0x77, dtype=torch.int64, device="cuda")
    pos = torch.full((T + pad,), -99, dtype=torch.int32, device="cuda")
    svr.moe_tree_plan(tree, dev(np.asarray(lens, np.int32)), mask, pos)
    got, gp = mask.cpu().numpy().view(np.uint64), pos.cpu().numpy()
    want, wp, on = to.plan(offsets, parents, lens, max_rows, words)
    assert np.array_equal(got[:T][on], want[on]) and np.array_equal(gp[:T][on], wp[on])
    # Rows from max_rows on and rows of no sequence stay as they were.
    off = np.concatenate([~on, np.ones(pad, bool)])
    assert (got[off] == 0x77).all() and (gp[off] == -99).all()
    # One output alone.
    only = torch.zeros_like(pos)
    svr.moe_tree_plan(tree, dev(np.asarray(lens, np.int32)), None, only)
    assert np.array_equal(only.cpu().numpy()[:T][on], wp[on])
    m2 = torch.zeros_like(mask)
    svr.moe_tree_plan(tree, None, m2, None)
    assert np.array_equal(m2.cpu().numpy().view(np.uint64)[:T][on], want[on])
    return want


@pytest.mark.parametrize("rows,kids,max_rows", [
    ([1], 1, 1), ([2], 1, 2), ([7], 3, 64), ([64], 8, 64), ([65], 4, 65), ([61, 0, 3, 128, 1], 5, 128),
    ([300, 17], 10, 300), ([1024], 30, 1024), ([40, 90, 70], 4, 70),
])
def test_plan_of_trees(rows, kids, max_rows):
    rng = np.random.default_rng(sum(rows))
    offsets, parents = forest(rows, kids, rng, level_order=kids != 5)
    check_plan(offsets, parents, [n + int(rng.integers(0, 60000)) for n in rows], max_rows)


def test_plan_of_chains_and_deep_trees():
    check_plan(np.array([0, 4]), None, [60004], 4)
    check_plan(np.array([0, 1024, 1030]), None, [1024, 9], 1024)          # ten rounds of doubling
    check_plan(np.array([0, 200]), np.arange(-1, 199), [500], 200, words=7)  # the same by parents; spare words


def test_plan_of_rows_that_hang_on_nothing():
    """Parents at or behind the row, negative or far out: roots of their own."""
    rng = np.random.default_rng(4)
    parents = np.array(random_parents(30, 3, rng), np.int32)
    parents[[5, 9, 17, 20]] = [5, 29, -1, 2 ** 31 - 1]
    parents[0] = 12  # not read
    parents[11] = -2 ** 31
    check_plan(np.array([0, 30]), parents, [30], 30)


def test_plan_of_many_sequences():
    rng = np.random.default_rng(5)
    rows = rng.integers(0, 9, 3000)
    offsets, parents = forest(rows, 2, rng)
    check_plan(offsets, parents, rows + rng.integers(0, 100, 3000), 8)


# ---- attention

class TreePlan(Plan):
    """A Plan whose new rows are trees."""

    def __init__(self, lay, rows, lens, rng, kids=3, words=None, **kw):
        super().__init__(lay, rows, lens, rng, **kw)
        _, parents = forest([int(r) for r in rows], kids, rng)
        words = words or -(-self.max_rows // 64)
        mask, pos, _ = to.plan(self.offsets, parents, self.lens, self.max_rows, words)
        self.parents, self.positions = parents, pos
        self.mask = np.concatenate([mask, np.full((self.T - len(mask), words), 2 ** 64 - 1, np.uint64)])


def check_tree(lay, plan, cache, dtype, rng, scale=None, q=None, ws=None):
    T = plan.T
    qt, q64 = rounded(rng.standard_normal((T, lay.heads, lay.dim)), dtype) if q is None else q
    out = torch.full((T, lay.heads, lay.dim), 77.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.full((T, lay.heads), 77.0, device="cuda")
    svr.moe_kv_tree_attention(desc_of(lay, scale or 0.0), plan.batch(), as_words(plan.mask), qt, dev(cache), out, lse,
                              ws=ws)
    torch.cuda.synchronize()
    ref, rl, size, reach, seen = to.attention(lay, cache, plan.offsets, plan.lens, plan.table, q64, plan.mask,
                                              plan.max_rows, scale)
    got, g = out.double().cpu().numpy(), lse.double().cpu().numpy()
    on = ~np.isnan(ref).any((1, 2))
    assert (got[~on] == 77).all() and (g[~on] == 77).all()
    tol = attention_tolerance(dtype, ref, size, reach, seen, lay.dim)[on]
    err = np.abs(got[on] - ref[on])
    assert np.all(err <= tol), (np.nanmax(err - tol), np.nanmax(err))
    empty = np.isneginf(rl[on])
    assert np.array_equal(np.isneginf(g[on]), empty)
    # The score's roundings, the weights' sum (a rounding for each token), the logarithm and its sum.
    u, r = 2.0 ** -24, rl[on]
    t = (lay.dim + 4) * u * reach[on] + (64 + seen[on, None]) * u + 8 * u * np.abs(np.where(empty, 0, r))
    assert np.all(np.abs(g[on][~empty] - r[~empty]) <= t[~empty])
    return got, ref


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,heads,kv_heads,page,window", [
    (64, 4, 4, 16, 0), (128, 8, 2, 32, 0), (192, 16, 1, 64, 0), (256, 10, 2, 16, 0),
    (192, 32, 2, 16, 7), (128, 5, 1, 64, 100), (64, 64, 1, 128, 3), (256, 16, 1, 32, 64),
])
def test_tree_attention_batches(dtype, dim, heads, kv_heads, page, window):
    log(f"tree attention {dtype} D={dim} {heads}/{kv_heads} page={page} W={window}")
    rng = np.random.default_rng(dim * heads + page)
    lay = ko.Layout(heads, kv_heads, dim, page, window)
    # A root alone on nothing, trees on short, long and no prefixes, no rows, rows before place 0.
    plan = TreePlan(lay, [1, 9, 0, 13, 7, 6, 2], [1, 9, 9, 130, 257, 4, 0], rng, pad_rows=3)
    got, _ = check_tree(lay, plan, plan.filled_cache(rng), dtype, rng)
    assert not got[plan.offsets[6]:plan.offsets[7]].any()  # an empty sequence


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 63, 64, 65, 100, 130])
@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 45])
def test_tree_rows_over_tiles(rows, prefix):
    """Masks of one word and more; new rows that begin at, before and behind a tile's border."""
    rng = np.random.default_rng(rows * 100 + prefix)
    lay = ko.Layout(2, 1, 64, 16)
    plan = TreePlan(lay, [rows], [prefix + rows], rng, kids=4)
    check_tree(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("window", [1, 2, 5, 31, 40, 64, 2 ** 31 - 1])
def test_window_counts_over_what_a_row_sees(window):
    """Windows shorter than a row's path, and longer: prefix tokens count by place, marked rows by their order."""
    rng = np.random.default_rng(window % 1000)
    lay = ko.Layout(4, 2, 64, 16, window)
    plan = TreePlan(lay, [70, 5, 40], [100, 300, 41], rng, kids=1)  # chains: paths of up to 70 rows
    check_tree(lay, plan, plan.filled_cache(rng), "f32", rng)
    plan = TreePlan(lay, [70, 5, 90], [100, 300, 91], rng, kids=3, words=3)
    check_tree(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("window", [0, 4])
def test_masks_that_are_no_trees(window):
    """Any bits: rows that see nothing, not themselves, rows behind them, bits behind the sequence's rows."""
    rng = np.random.default_rng(21)
    lay = ko.Layout(4, 2, 128, 16, window)
    plan = TreePlan(lay, [40, 3, 70], [40, 50, 70], rng, pad_rows=1)
    plan.mask = rng.integers(0, 2 ** 64, plan.mask.shape, dtype=np.uint64) & rng.integers(
        0, 2 ** 64, plan.mask.shape, dtype=np.uint64)
    plan.mask[[0, 7, 41]] = 0
    plan.mask[8] = 2 ** 64 - 1
    got, _ = check_tree(lay, plan, plan.filled_cache(rng), "bf16", rng)
    assert not got[[0, 7]].any() and got[41].any()  # no prefix, a prefix


def test_a_chain_gives_what_causal_attention_gives():
    """Each lies within its bound of the exact result, so they differ by two of them at most (the tokens of a
    tree may be cut otherwise than those of a batch)."""
    rng = np.random.default_rng(22)
    for lay, rows, lens, width in ((ko.Layout(16, 2, 192, 64), [4], [900], None), (ko.Layout(8, 2, 64, 16), [4, 1], [333, 90], None),
                                   (ko.Layout(10, 1, 128, 64), [4], [2000], 700)):
        plan = TreePlan(lay, rows, lens, rng, kids=1, width=width)
        cache = plan.filled_cache(rng)
        for dtype in ("bf16", "f32"):
            q, q64 = rounded(rng.standard_normal((plan.T, lay.heads, lay.dim)), dtype)
            c, a, b = dev(cache), torch.empty_like(q), torch.empty_like(q)
            svr.moe_kv_attention(desc_of(lay), plan.batch(), q, c, a)
            svr.moe_kv_tree_attention(desc_of(lay), plan.batch(), as_words(plan.mask), q, c, b)
            ref, _, size, reach, seen = ko.attention(lay, cache, plan.offsets, plan.lens, plan.table, q64)
            tol = attention_tolerance(dtype, ref, size, reach, seen, lay.dim)
            assert np.all(np.abs(a.double().cpu().numpy() - b.double().cpu().numpy()) <= 2 * tol)


@pytest.mark.parametrize("rows,length,heads,kv_heads,width", [
    (7, 900, 16, 1, 2000), (24, 2500, 64, 4, None), (40, 3000, 32, 2, None), (61, 1500, 32, 4, 3000),
    (130, 1500, 16, 1, None), (300, 900, 8, 2, 400), (9, 3000, 48, 3, 900), (20, 2000, 16, 8, 700),
])
def test_one_tree_however_its_tokens_are_cut(rows, length, heads, kv_heads, width):
    """Row tiles of one and two, parts of four and eight waves, joined by the last workgroup or a second
    kernel, more than run at once; tables longer than the tokens."""
    log(f"one tree {rows} rows, {length} tokens, {heads}/{kv_heads}, table of {width}")
    rng = np.random.default_rng(rows)
    lay = ko.Layout(heads, kv_heads, 64, 32)
    plan = TreePlan(lay, [rows], [length], rng, kids=4, width=width)
    check_tree(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("dtype,dim", [("bf16", 192), ("f32", 64), ("f16", 128), ("bf16", 256)])
@pytest.mark.parametrize("lens,width", [([2900], None), ([2900], 700), ([1800, 333], 700)])
def test_tree_attention_over_many_tokens(dtype, dim, lens, width):
    """Every way in which tokens are cut and joined."""
    log(f"long {dtype} D={dim} {lens} {width}")
    rng = np.random.default_rng(dim + len(lens))
    lay = ko.Layout(10, 1, dim, 64)
    plan = TreePlan(lay, [9] * len(lens), lens, rng, width=width)
    check_tree(lay, plan, plan.filled_cache(rng), dtype, rng)
    lay.window = 700
    check_tree(lay, plan, plan.filled_cache(rng), dtype, rng)


@pytest.mark.parametrize("seqs,heads,kv_heads,window", [(64, 4, 2, 0), (65, 6, 3, 0), (150, 2, 1, 0), (70, 3, 1, 120)])
def test_tree_attention_over_uneven_sequences(seqs, heads, kv_heads, window):
    log(f"uneven {seqs} {heads}/{kv_heads} W={window}")
    rng = np.random.default_rng(seqs)
    lay = ko.Layout(heads, kv_heads, 64, 16, window)
    rows = rng.integers(0, 12, seqs)
    lens = rows + rng.integers(0, 90, seqs)
    rows[seqs // 2], lens[seqs // 2] = 41, 2100
    rows[-1], lens[-1] = 2, 700
    plan = TreePlan(lay, list(rows), list(lens), rng, pad_rows=1)
    check_tree(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,heads,kv_heads,longest,window", [
    (30, 16, 4, 4000, 0), (30, 16, 4, 4000, 3500), (70, 8, 4, 4000, 0), (6, 16, 16, 4000, 0),
])
def test_trees_of_which_more_than_run_at_once(dtype, seqs, heads, kv_heads, longest, window):
    """Parts of the mean of uneven sequences, and even ones that are not cut."""
    log(f"more than at once {dtype} {seqs} {heads}/{kv_heads} W={window}")
    rng = np.random.default_rng(seqs + window)
    lay = ko.Layout(heads, kv_heads, 64, 16, window)
    rows = rng.integers(1, 27, seqs)
    lens = rows + rng.integers(0, 900, seqs)
    rows[seqs // 2], lens[seqs // 2], lens[0], lens[-1] = 26, longest, 2500, 27
    plan = TreePlan(lay, list(rows), list(lens), rng)
    check_tree(lay, plan, plan.filled_cache(rng), dtype, rng)
    if seqs == 6:
        plan = TreePlan(lay, [26] * seqs, [700] * seqs, rng, width=300)
        check_tree(lay, plan, plan.filled_cache(rng), dtype, rng)


def test_tree_attention_hides_pages_that_are_not_there():
    rng = np.random.default_rng(23)
    lay = ko.Layout(4, 2, 128, 16)
    plan = TreePlan(lay, [9, 5], [100, 40], rng)
    cache = plan.filled_cache(rng)
    plan.table[0, 2], plan.table[0, 6], plan.table[1, 0] = -1, plan.n_pages, 2 ** 31 - 1  # (places 96 on: new rows)
    cache[0] = 0xFF
    for b in range(2):
        plan.table[b][plan.table[b] == 0] = -7
    check_tree(lay, plan, cache, "bf16", rng)
    plan.table[:] = -1
    got, _ = check_tree(lay, plan, cache, "f32", rng)
    assert not got.any()


def test_tree_attention_lengths_beyond_the_table():
    rng = np.random.default_rng(24)
    lay = ko.Layout(2, 1, 64, 16)
    plan = TreePlan(lay, [6, 6], [34, 64], rng, width=2)
    check_tree(lay, plan, plan.filled_cache(rng), "f32", rng)


def test_tree_attention_leaves_rows_beyond_max_rows():
    rng = np.random.default_rng(25)
    lay = ko.Layout(2, 1, 64, 16, 9)
    plan = TreePlan(lay, [70, 5], [90, 20], rng, words=2)
    plan.mask |= np.uint64(1 << 20)
    plan.max_rows = 66
    check_tree(lay, plan, plan.filled_cache(rng), "bf16", rng)


def test_a_row_that_is_not_finite_is_nan_for_those_who_see_it():
    rng = np.random.default_rng(26)
    lay = ko.Layout(4, 2, 64, 16)
    parents = np.array([-1, 0, 0, 1, 2, 2], np.int32)
    plan = TreePlan(lay, [6], [30], rng)
    plan.mask, _, _ = to.plan([0, 6], parents, [30], 6, 1)
    q, _ = rounded(rng.standard_normal((6, 4, 64)), "bf16")
    k, v = (rng.standard_normal((6, 2, 64)).astype(np.float32) for _ in "kv")
    k[2, 1, 3] = np.inf
    cache = dev(plan.filled_cache(rng))
    svr.moe_kv_append(desc_of(lay), plan.batch(), None, dev(k), dev(v), cache, None)
    out = torch.empty_like(q)
    svr.moe_kv_tree_attention(desc_of(lay), plan.batch(), as_words(plan.mask), q, cache, out)
    bad = torch.isnan(out).cpu().numpy()
    assert bad[[2, 4, 5], 2:].all() and not bad[[0, 1, 3]].any() and not bad[:, :2].any()


def test_tree_and_causal_calls_on_one_workspace():
    rng = np.random.default_rng(27)
    cases = []
    for lay, rows, lens, dtype, width in (
            (ko.Layout(8, 1, 192, 16), [5], [900], "bf16", None), (ko.Layout(8, 2, 64, 16), [9, 2], [700, 90], "f32", 400),
            (ko.Layout(16, 2, 128, 32), [7] * 30, list(range(7, 7 + 42 * 30, 42)), "f16", None)):
        plan = TreePlan(lay, rows, lens, rng, width=width)
        q, _ = rounded(rng.standard_normal((plan.T, lay.heads, lay.dim)), dtype)
        cases.append((desc_of(lay), plan.batch(), as_words(plan.mask), q, dev(plan.filled_cache(rng))))
    n = max(svr.moe_kv_attention_workspace_bytes(d, b, len(q)) for d, b, _, q, _ in cases)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:16384].zero_()
    want = []
    for d, b, m, q, c in cases:
        out = torch.empty_like(q)
        svr.moe_kv_tree_attention(d, b, m, q, c, out)
        want.append(out)
    for i in (0, 1, 2, 2, 1, 0, 0, 2):
        d, b, m, q, c = cases[i]
        out = torch.full_like(q, float("nan"))
        svr.moe_kv_tree_attention(d, b, m, q, c, out, ws=ws)
        assert torch.equal(out, want[i]) and not ws[:16384].any(), i
        svr.moe_kv_attention(d, b, q, c, out, ws=ws)
        assert not ws[:16384].any(), i


# ---- commit

def check_commit(lay, rows, lens, paths, n_accepted, rng, layers=1, max_rows=None, wide=None, **kw):
    plan = Plan(lay, rows, lens, rng, **kw)
    if max_rows:
        plan.max_rows = max_rows
    wide = wide or max(len(p) for p in paths)
    path = np.full((len(paths), wide), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    shape = (layers, plan.n_pages, lay.kv_heads, lay.page_bytes)
    caches = rng.integers(0, 256, shape).astype(np.uint8)
    got, kept = [dev(c) for c in caches], torch.full((len(rows),), -9, dtype=torch.int32, device="cuda")
    svr.moe_kv_commit(desc_of(lay), plan.batch(), dev(path), dev(np.asarray(n_accepted, np.int32)), got, kept)
    for g, c in zip(got, caches):
        want_kept = to.commit(lay, c, plan.offsets, plan.lens, plan.table, plan.max_rows, path, n_accepted)
        assert np.array_equal(g.cpu().numpy(), c)
    assert np.array_equal(kept.cpu().numpy(), want_kept)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("page,layers", [(16, 3), (64, 1)])
def test_commit_of_paths(dim, page, layers):
    rng = np.random.default_rng(dim + page)
    lay = ko.Layout(6, 3, dim, page)
    rows, lens = [9, 0, 1, 20, 12, 6], [9, 5, 40, 70, 64 + 12, 3]
    paths = [[0, 1, 2, 3], [0], [0], [0, 2, 3, 4, 11, 19], [0, 5, 11], [0, 4, 5]]  # overlapping; over a page's end
    check_commit(lay, rows, lens, paths, [3, 0, 0, 5, 2, 2], rng, layers)


def test_commit_of_long_paths():
    """More tokens than a workgroup moves at a time, from places that it writes."""
    rng = np.random.default_rng(31)
    lay = ko.Layout(2, 1, 256, 16)
    rows, paths = [], []
    for n in (300, 65, 200):
        rows.append(n)
        paths.append([0] + sorted(rng.choice(np.arange(1, n), n * 2 // 3, replace=False).tolist()))
    check_commit(lay, rows, [r + 33 for r in rows], paths, [len(p) - 1 for p in paths], rng)


def test_commit_of_what_is_no_path():
    """Counts and entries out of range, rows beyond max_rows: nothing but the sequences' own rows moves."""
    rng = np.random.default_rng(32)
    lay = ko.Layout(2, 2, 128, 16)
    check_commit(lay, [8, 8, 8, 8], [30, 30, 30, 30], [[0, 9, 2 ** 31 - 1, -5], [0, 2, 3, 4], [0, 0, 5, 1], [0, 6, 7, 3]],
                 [3, 100, -7, 2], rng)
    check_commit(lay, [8, 2], [30, 31], [[0, 3, 6, 7], [0, 1, 1, 1]], [3, 3], rng, max_rows=7)
    check_commit(lay, [8], [30], [[0]], [4], rng)                 # a path of the root alone
    check_commit(lay, [8, 8], [5, 40], [[0, 4, 6], [0, 5, 7]], [2, 2], rng, width=2)  # before place 0, beyond the table


def test_commit_of_many_sequences_and_layers():
    rng = np.random.default_rng(33)
    lay = ko.Layout(2, 2, 64, 16)
    rows = rng.integers(1, 12, 90)
    paths = [[0] + sorted(rng.choice(np.arange(1, r), min(int(rng.integers(0, 5)), r - 1), replace=False).tolist())
             for r in rows]
    check_commit(lay, list(rows), list(rows + rng.integers(0, 40, 90)), paths, [len(p) - 1 for p in paths], rng,
                 layers=6, wide=11)


def test_commit_of_layers_side_by_side():
    """All layers' caches in one tensor, in any order, with no room between; overlapping ones are refused."""
    rng = np.random.default_rng(35)
    lay = ko.Layout(2, 2, 64, 16)
    plan = Plan(lay, [9], [40], rng)
    batch = plan.batch()
    path, n = dev(np.array([[0, 3, 8]], np.int32)), dev(np.array([2], np.int32))
    start = dev(rng.integers(0, 256, (3, plan.n_pages, 2, lay.page_bytes)).astype(np.uint8))
    one, all_ = start.clone(), start.clone()
    for c in one:
        svr.moe_kv_commit(desc_of(lay), batch, path, n, [c])
    svr.moe_kv_commit(desc_of(lay), batch, path, n, [all_[2], all_[0], all_[1]])
    torch.cuda.synchronize()
    assert torch.equal(one, all_) and not torch.equal(one, start)
    pages = all_.view(-1, 2, lay.page_bytes)
    with pytest.raises(svr.MoeError):
        svr.moe_kv_commit(desc_of(lay), batch, path, n, [pages[:plan.n_pages], pages[1:plan.n_pages + 1]])


def test_plan_and_commit_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(34)
    lay = ko.Layout(2, 1, 64, 16)
    plan = Plan(lay, [9, 7], [40, 30], rng)
    offsets, parents = forest([9, 7], 2, rng)
    tree, batch = tree_of(offsets, parents, 9, 2), plan.batch()
    lens = batch.seq_lens
    path = dev(np.array([[0, 3, 8], [0, 2, 5]], np.int32))
    n = dev(np.array([2, 2], np.int32))
    start = dev(rng.integers(0, 256, (plan.n_pages, 1, lay.page_bytes)).astype(np.uint8))
    cache = start.clone()
    mask = torch.empty((16, 1), dtype=torch.int64, device="cuda")
    pos, kept = torch.empty(16, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")

    def step(stream=None):
        svr.moe_tree_plan(tree, lens, mask, pos, stream=stream)
        svr.moe_kv_commit(desc_of(lay), batch, path, n, [cache], kept, stream=stream)

    def outputs():
        torch.cuda.synchronize()
        got = [t.clone() for t in (mask, pos, kept, cache)]
        for t in (mask, pos, kept):
            t.fill_(-1)
        cache.copy_(start)
        torch.cuda.synchronize()
        return got

    step()
    first = outputs()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(side)
    assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    with torch.cuda.graph(g, stream=side):
        step()
    outputs()
    for k in range(3):
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    # New lengths and paths in place: the graph follows them.
    lens.add_(1)
    path[:, 1] += 1
    step()
    second = outputs()
    assert torch.equal(second[2], first[2] + 1)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(second, outputs()))


def test_trees_in_a_cache_beyond_four_gibibytes():
    """The last pages of a cache of 4.5 GB, one and two row tiles a wave: attention and commit."""
    rng = np.random.default_rng(36)
    lay = ko.Layout(8, 8, 128, 1024)
    n = 4000
    assert (n - 2) * 8 * lay.page_bytes > 2 ** 32
    big = svr.kv_cache(desc_of(lay), n)
    for rows, width in ((5, 2), (40, 16)):
        plan = TreePlan(lay, [rows], [1500], rng, width=width, spare=0)
        small = plan.filled_cache(rng)
        table = np.full((1, width), -1, np.int32)
        for j in range(2):
            table[0, j] = n - 1 - j
            big[n - 1 - j] = dev(small[plan.table[0, j]])
        batch = svr.KvBatch(dev(plan.offsets), dev(plan.lens), dev(table), rows)
        q = rounded(rng.standard_normal((rows, 8, 128)), "bf16")
        out, _ = check_tree(lay, plan, small, "bf16", rng, q=q)
        got = torch.empty_like(q[0])
        svr.moe_kv_tree_attention(desc_of(lay), batch, as_words(plan.mask), q[0], big, got)
        path, kept = np.array([[0, 2, 4]], np.int32), torch.empty(1, dtype=torch.int32, device="cuda")
        svr.moe_kv_commit(desc_of(lay), batch, dev(path), dev(np.array([2], np.int32)), [big], kept)
        to.commit(lay, small, plan.offsets, plan.lens, plan.table, rows, path, [2])
        assert np.array_equal(got.double().cpu().numpy(), out)
        for j in range(2):
            assert np.array_equal(big[n - 1 - j].cpu().numpy(), small[plan.table[0, j]])
        assert int(kept[0]) == 1500 - rows + 3


def test_tree_attention_of_rows_apart_on_two_streams_and_in_a_graph():
    """Views of a fused projection; calls at once on workspaces of their own; replays follow masks and lengths."""
    rng = np.random.default_rng(37)
    lay = ko.Layout(16, 2, 128, 16)
    plan = TreePlan(lay, [21, 4], [900, 260], rng)
    T, d, batch = plan.T, desc_of(lay), plan.batch()
    cache = plan.filled_cache(rng)
    t, q64 = rounded(rng.standard_normal((T, 16, 128)), "bf16")
    fused = torch.full((T, 20, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 3:19] = t
    q = fused[:, 3:19]
    want, _ = check_tree(lay, plan, cache, "bf16", rng, q=(q, q64))
    gpu, mask, lens = dev(cache), as_words(plan.mask), batch.seq_lens
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [svr.kv_workspace(d, batch, T) for _ in streams]
    outs = [torch.empty((T, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, w, st in zip(outs, ws, streams):
            svr.moe_kv_tree_attention(d, batch, mask, q, gpu, o, ws=w, stream=st)
    torch.cuda.synchronize()
    assert all(np.array_equal(o.double().cpu().numpy(), want) for o in outs)

    g, out = torch.cuda.CUDAGraph(), outs[0]
    with torch.cuda.graph(g, stream=streams[0]):
        svr.moe_kv_tree_attention(d, batch, mask, q, gpu, out, ws=ws[0])
    own = to.plan(plan.offsets, None, plan.lens, plan.max_rows, plan.mask.shape[1])[0]  # chains
    for new_mask, new_lens in ((plan.mask, plan.lens), (own, plan.lens), (own, plan.lens - [17, 250]),
                               (plan.mask, plan.lens)):
        mask.copy_(as_words(new_mask))
        lens.copy_(dev(np.asarray(new_lens, np.int32)))
        svr.moe_kv_tree_attention(d, batch, mask, q, gpu, outs[1], ws=ws[1])
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, outs[1]) and not out.isnan().any()
    assert np.array_equal(out.double().cpu().numpy(), want)
