"""A verify step on trees of drafts without a GPU: the oracles against closed forms and brute force,
and what the library and its binding refuse before anything is enqueued."""

import ctypes
import itertools

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from speculative_verify_router_amd import _binding as B
from oracle import kv_oracle as ko, sample_oracle as so, tree_oracle as to
from tree_support import forest, random_parents

A = 1 << 20  # an aligned address that is never read: every call here is refused or empty


# ---- oracles

def test_masks_of_a_chain_are_causal():
    mask, pos, on = to.plan([0, 70], None, [100], 70, 2)
    assert on.all() and pos.tolist() == list(range(30, 100))
    for i in range(70):
        assert int(mask[i, 0]) + (int(mask[i, 1]) << 64) == (1 << (i + 1)) - 1


def test_masks_by_hand():
    #      0
    #    1   2      5: its parent is not an earlier row, so it hangs on nothing
    #  3   4        6 follows 5
    parents = [7, 0, 0, 1, 1, 5, 5]
    mask, pos, _ = to.plan([0, 7], parents, [10], 7, 1)
    assert [int(m) for m in mask[:, 0]] == [1, 3, 5, 11, 19, 32, 96]
    assert pos.tolist() == [3, 4, 4, 5, 5, 3, 4]
    assert to.children(parents, 0, 7, 0, 9) == [1, 2] and to.children(parents, 0, 7, 0, 1) == [1]


def test_tree_attention_of_a_chain_is_attention():
    rng = np.random.default_rng(1)
    for window in (0, 3, 9):
        lay = ko.Layout(4, 2, 64, 16, window)
        cache = rng.integers(0, 256, (4, 2, lay.page_bytes)).astype(np.uint8)
        for page in cache:
            for p in page:
                ko.page_parts(lay, p)[2][:] = 126
                ko.page_parts(lay, p)[3][:] = 127
        table, q = np.array([[2, 0, 3]], np.int32), rng.standard_normal((5, 4, 64))
        mask, _, _ = to.plan([0, 5], None, [37], 5, 1)
        a = ko.attention(lay, cache, [0, 5], [37], table, q)
        b = to.attention(lay, cache, [0, 5], [37], table, q, mask, 5)
        assert np.array_equal(a[4], b[4]) and np.allclose(a[0], b[0], rtol=1e-13, atol=1e-13)


def test_siblings_do_not_see_each_other():
    """A branch alone, appended as a chain, gives what the tree gives its rows."""
    rng = np.random.default_rng(2)
    lay = ko.Layout(2, 1, 64, 16)
    parents = [-1, 0, 0, 1, 2]
    cache = np.zeros((2, 1, lay.page_bytes), np.uint8)
    kv, q = rng.standard_normal((2, 9, 1, 64)), rng.standard_normal((5, 2, 64))
    table = np.array([[0, 1]], np.int32)
    ko.append(lay, cache, [0, 9], [9], table, np.zeros((9, 2, 64)), kv[0], kv[1])
    mask, _, _ = to.plan([0, 5], parents, [9], 5, 1)
    tree = to.attention(lay, cache, [0, 5], [9], table, q, mask, 5)[0]
    alone = np.zeros_like(cache)
    rows = [0, 1, 2, 3, 4, 6, 8]  # the prefix, the root, rows 2 and 4
    ko.append(lay, alone, [0, 7], [7], table, np.zeros((7, 2, 64)), kv[0][rows], kv[1][rows])
    chain = ko.attention(lay, alone, [0, 3], [7], table, q[[0, 2, 4]])[0]
    assert np.allclose(tree[[0, 2, 4]], chain, rtol=1e-13, atol=1e-13)


def test_commit_moves_a_path_in_order():
    rng = np.random.default_rng(3)
    lay = ko.Layout(2, 2, 64, 16)
    cache = rng.integers(0, 256, (3, 2, lay.page_bytes)).astype(np.uint8)
    was, table = cache.copy(), np.array([[1, 2]], np.int32)
    # Rows 1 and 2 of the path come from places that the path writes too.
    kept = to.commit(lay, cache, [0, 8], [20], table, 8, np.array([[0, 2, 3, 7, -1]]), [3])
    assert kept.tolist() == [16]
    for h, part in itertools.product(range(2), range(4)):
        def at(c, place):
            page, o = ko.slot(lay, table[0], 3, place)
            return ko.page_parts(lay, c[page, h])[part][o].tolist()
        assert [at(cache, 12 + i) for i in range(4)] == [at(was, 12 + r) for r in (0, 2, 3, 7)]
        assert [at(cache, p) for p in [*range(12), *range(16, 20)]] == [at(was, p) for p in [*range(12), *range(16, 20)]]


def exact_distribution(p, q, kids):
    """The first token's distribution when `kids` drafts are drawn from q and tried in turn, over all u."""
    out, w, reach = np.zeros_like(p), p.copy(), 1.0
    for _ in range(kids):
        # A draft x is accepted with min(1, w(x)/q(x)): over its draw, min(q, w).
        took = np.minimum(w, q)
        out += reach * took
        reach *= 1.0 - took.sum()
        left = np.maximum(w - q, 0.0)
        w = left / left.sum() if left.sum() > 0 else left
    return out + reach * w


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_drawn_drafts_leave_the_targets_distribution(kids):
    """The rule that the oracle follows gives p, whatever q is: in closed form, and by counting."""
    rng = np.random.default_rng(kids)
    p, q = rng.dirichlet(np.ones(6)), rng.dirichlet(np.ones(6))
    assert np.allclose(exact_distribution(p, q, kids), p, atol=1e-14)
    n, V = 4000, 6
    rows = 1 + kids
    logits = np.log(np.broadcast_to(p, (rows, V)))
    parents = [-1] + [0] * kids
    count = np.zeros(V)
    for _ in range(n):
        tokens = np.concatenate([[0], rng.choice(V, kids, p=q)])
        got = so.verify(logits, [0, rows], parents, tokens, rng.random(rows), rng.random(1), rows, kids,
                        np.broadcast_to(q, (rows, V)))
        count[got["accepted"][0][0]] += 1
    # Five standard deviations of a count, of each of six tokens.
    assert np.all(np.abs(count - n * p) <= 5 * np.sqrt(n * p * (1 - p)))


def test_given_drafts_leave_the_targets_distribution():
    """u over a fine grid: token t of the drafts is accepted in a share p(t) of it, the rest follows p."""
    p = np.array([0.4, 0.1, 0.05, 0.25, 0.2])
    tokens, parents = [9, 3, 1, 3], [-1, 0, 0, 0]  # token 3 twice: the second has nothing left
    count = np.zeros(5)
    grid = (np.arange(20) + 0.5) / 20
    for u1, u2, us in itertools.product(grid, grid, grid):
        got = so.verify(np.log(np.broadcast_to(p, (4, 5))), [0, 4], parents, tokens, [0, u1, u2, 0.0], [us], 4, 3)
        count[got["accepted"][0][0]] += 1
    # Each border moves a share by at most one grid cell.
    assert np.all(np.abs(count / 8000 - p) <= 0.05)
    assert abs(count[3] / 8000 - 0.25) < 1e-12  # (a whole number of cells)


def test_the_share_taken_off_grows_by_what_is_left():
    """(p - c q)+ with c = 1, then c + S, is what normalising after every rejection gives."""
    rng = np.random.default_rng(5)
    p, q = rng.dirichlet(np.ones(50)), rng.dirichlet(np.ones(50))
    w, c, s = p.copy(), 0.0, 1.0
    for _ in range(5):
        w = np.maximum(w - q, 0.0)
        if w.sum() == 0:
            break
        w /= w.sum()
        c += s
        v = np.maximum(p - c * q, 0.0)
        s = v.sum()
        assert np.allclose(w, v / s, rtol=1e-9, atol=1e-12)


def test_greedy_sampling_is_verify_accept():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((4, 30))
    best = x.argmax(1)
    got = so.verify(x, [0, 4], None, [0, best[0], best[1], (best[2] + 1) % 30], rng.random(4), [0.5], 4, 1,
                    temperature=[0.0])
    assert got["accepted"][0] == [best[0], best[1], best[2], -1] and got["path"][0] == [0, 1, 2, -1]


def test_rows_without_a_distribution():
    x = np.full((2, 7), -np.inf)
    assert so.verify(x, [0, 2], None, [0, 3], [0, 0.0], [0.5], 2, 1)["accepted"][0] == [-1, -1]
    x[0, 2], x[0, 4] = np.nan, np.inf
    assert so.verify(x, [0, 2], None, [0, 4], [0, 0.9], [0.5], 2, 1)["accepted"][0] == [4, -1]


# ---- refusals

def tree_c(**kw):
    a = dict(n_seqs=2, n_rows=10, max_rows=6, max_children=3, q_offsets=A, parents=A)
    a.update(kw)
    return ctypes.byref(B._Tree(*a.values()))


def plan_status(**kw):
    a = dict(tree=tree_c(), lens=A, mask=A, words=1, pos=A, stream=None)
    a.update(kw)
    return svr.lib().moe_tree_plan(*a.values())


TREE_OUT_OF_RANGE = [dict(n_seqs=-1), dict(n_seqs=65537), dict(n_rows=-1), dict(n_rows=65537), dict(max_rows=0),
                     dict(max_rows=1025), dict(max_children=0), dict(max_children=1025)]


def test_plan_refusals():
    for kw in TREE_OUT_OF_RANGE:
        assert plan_status(tree=tree_c(**kw)) == B.ERR_SHAPE, kw
    for kw, status in [
        (dict(tree=None), B.ERR_NULL), (dict(tree=tree_c(q_offsets=None)), B.ERR_NULL),
        (dict(tree=tree_c(q_offsets=A + 2)), B.ERR_ARG), (dict(tree=tree_c(parents=A + 1)), B.ERR_ARG),
        (dict(lens=None), B.ERR_NULL), (dict(words=0), B.ERR_SHAPE), (dict(words=17), B.ERR_SHAPE),
        (dict(tree=tree_c(max_rows=65)), B.ERR_SHAPE), (dict(mask=A + 4), B.ERR_ARG), (dict(pos=A + 2), B.ERR_ARG),
        (dict(lens=A + 1), B.ERR_ARG),
    ]:
        assert plan_status(**kw) == status, kw
    assert plan_status(mask=None, words=0, pos=None) == B.OK
    assert plan_status(tree=tree_c(n_rows=0)) == B.OK
    assert plan_status(tree=tree_c(n_seqs=0, q_offsets=None)) == B.OK


def kv_desc(**kw):
    a = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=64)
    a.update(kw)
    return svr.KvDesc(**a)


def kv_batch(**kw):
    a = dict(n_seqs=2, n_tokens=10, max_rows=6, pages_per_seq=100, q_offsets=A, seq_lens=A, page_table=A)
    a.update(kw)
    return ctypes.byref(B._KvBatch(*a.values()))


def attention_status(**kw):
    a = dict(desc=kv_desc(), batch=kv_batch(), dtype=B.BF16, mask=A, words=1, q=A, qs=1024, cache=A, pages=9, out=A,
             lse=A, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    a["desc"] = a["desc"].c()
    return svr.lib().moe_kv_tree_attention(*a.values())


def test_tree_attention_refusals():
    for kw, status in [
        (dict(mask=None), B.ERR_NULL), (dict(mask=A + 4), B.ERR_ARG), (dict(words=0), B.ERR_SHAPE),
        (dict(words=17), B.ERR_SHAPE), (dict(batch=kv_batch(max_rows=65)), B.ERR_SHAPE),
        (dict(batch=kv_batch(max_rows=1025), words=16), B.ERR_SHAPE),
        (dict(dtype=B.Q4_K), B.ERR_DTYPE), (dict(q=None), B.ERR_NULL), (dict(out=None), B.ERR_NULL),
        (dict(cache=None), B.ERR_NULL), (dict(qs=1000), B.ERR_SHAPE), (dict(pages=0), B.ERR_SHAPE),
        (dict(q=A + 1), B.ERR_ARG), (dict(out=A + 1), B.ERR_ARG), (dict(cache=A + 8), B.ERR_ARG),
        (dict(lse=A + 2), B.ERR_ARG), (dict(ws=None), B.ERR_NULL), (dict(ws=A + 128), B.ERR_ARG),
        (dict(ws_bytes=100), B.ERR_WORKSPACE), (dict(desc=kv_desc(head_dim=96)), B.ERR_SHAPE),
        (dict(batch=kv_batch(seq_lens=None)), B.ERR_NULL), (dict(batch=None), B.ERR_NULL),
    ]:
        assert attention_status(**kw) == status, kw
    for b in (kv_batch(n_tokens=0), kv_batch(max_rows=0), kv_batch(n_seqs=0, q_offsets=None, seq_lens=None,
                                                                  page_table=None)):
        assert attention_status(batch=b, mask=None) == B.OK


def commit_status(**kw):
    caches = kw.pop("caches", (A,))
    a = dict(desc=kv_desc(), batch=kv_batch(), path=A, stride=6, n=A,
             caches=None if caches is None else (ctypes.c_void_p * max(len(caches), 1))(*caches),
             n_caches=len(caches or ()), pages=9, kept=A + 64, stream=None)
    a.update(kw)
    a["desc"] = a["desc"].c()
    return svr.lib().moe_kv_commit(*a.values())


def test_commit_refusals():
    for kw, status in [
        (dict(path=None), B.ERR_NULL), (dict(n=None), B.ERR_NULL), (dict(caches=None, n_caches=1), B.ERR_NULL),
        (dict(caches=(A, None)), B.ERR_NULL), (dict(caches=(A, A + 8)), B.ERR_ARG), (dict(caches=(A, A + 64, A)), B.ERR_ARG), (dict(caches=()), B.ERR_SHAPE),
        (dict(caches=[A + 64 * i for i in range(257)]), B.ERR_SHAPE), (dict(stride=0), B.ERR_SHAPE), (dict(pages=0), B.ERR_SHAPE),
        (dict(path=A + 2), B.ERR_ARG), (dict(n=A + 1), B.ERR_ARG), (dict(kept=A + 2), B.ERR_ARG), (dict(kept=A), B.ERR_ARG),
        (dict(n=A + 64), B.ERR_ARG),  # kept_lens
        (dict(caches=(A + 1024, A, A + 9 * 2 * kv_desc().page_bytes - 16)), B.ERR_ARG),  # pages of the first two
        (dict(batch=None), B.ERR_NULL), (dict(batch=kv_batch(page_table=None)), B.ERR_NULL),
        (dict(batch=kv_batch(pages_per_seq=0)), B.ERR_SHAPE), (dict(desc=kv_desc(page_size=17)), B.ERR_SHAPE),
        (dict(desc=kv_desc(n_heads=1024, n_kv_heads=1024), batch=kv_batch(n_seqs=16384)), B.ERR_SHAPE),
    ]:
        assert commit_status(**kw) == status, kw
    assert commit_status(batch=kv_batch(n_seqs=0, q_offsets=None, seq_lens=None, page_table=None)) == B.OK


def sample_status(**kw):
    a = dict(tree=tree_c(), x=A, dtype=B.F32, V=1000, stride=1000, tokens=A, q=A, qs=1000, temp=A, au=A, su=A, vh=A,
             h=8, accepted=A, path=A, n=A, pending=A, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return svr.lib().moe_verify_sample(*a.values())


def test_sample_refusals():
    for kw in TREE_OUT_OF_RANGE + [dict(n_rows=16385), dict(n_seqs=16385)]:
        assert sample_status(tree=tree_c(**kw)) == B.ERR_SHAPE, kw
    for kw, status in [
        (dict(V=0), B.ERR_SHAPE), (dict(V=2 ** 30 + 1, stride=2 ** 31, qs=2 ** 31), B.ERR_SHAPE),
        (dict(stride=999), B.ERR_SHAPE), (dict(qs=999), B.ERR_SHAPE), (dict(h=-1), B.ERR_SHAPE),
        (dict(vh=None, pending=None), B.ERR_SHAPE), (dict(vh=None, h=0), B.ERR_NULL), (dict(pending=None), B.ERR_NULL),
        (dict(dtype=B.Q8_0), B.ERR_DTYPE), (dict(tree=None), B.ERR_NULL), (dict(tree=tree_c(q_offsets=None)), B.ERR_NULL),
        *[({k: None}, B.ERR_NULL) for k in ("x", "tokens", "au", "su", "accepted", "n", "ws")],
        (dict(ws_bytes=131072), B.ERR_WORKSPACE), (dict(ws=A + 64), B.ERR_ARG), (dict(x=A + 2), B.ERR_ARG),
        (dict(dtype=B.BF16, x=A + 1), B.ERR_ARG),
        *[({k: A + 2}, B.ERR_ARG) for k in ("tokens", "q", "temp", "au", "su", "vh", "accepted", "path", "n", "pending")],
    ]:
        assert sample_status(**kw) == status, kw
    assert sample_status(tree=tree_c(n_rows=0)) == B.OK
    assert sample_status(tree=tree_c(n_seqs=0, q_offsets=None)) == B.OK
    out = ctypes.c_size_t()
    f = svr.lib().moe_sample_workspace_bytes
    assert f(tree_c(), 1000, None) == B.ERR_NULL and f(None, 1000, ctypes.byref(out)) == B.ERR_NULL
    assert f(tree_c(), 0, ctypes.byref(out)) == B.ERR_SHAPE
    assert f(tree_c(q_offsets=None, parents=None), 1000, ctypes.byref(out)) == B.OK and out.value > 131072


def test_sample_workspace_serves_every_smaller_batch():
    z = torch.zeros(2, dtype=torch.int32)
    t = svr.DraftTree(z, None, 4)
    for V in (131072, 5000, 1):
        most = svr.moe_sample_workspace_bytes(t, 600, V)
        for rows in (1, 2, 7, 64, 511, 600):
            assert svr.moe_sample_workspace_bytes(t, rows, V) <= most


def test_the_binding_refuses_what_it_cannot_pass_on():
    i32 = dict(dtype=torch.int32)
    z = torch.zeros(3, **i32)
    tree = svr.DraftTree(torch.tensor([0, 3], **i32), z, 3, 2)
    with pytest.raises(ValueError, match="parents: expected torch.int32"):
        svr.DraftTree(z, z.long(), 3)
    with pytest.raises(ValueError, match="parents: expected"):
        svr.DraftTree(z, z[None], 3)
    with pytest.raises(ValueError, match="q_offsets"):
        svr.DraftTree(z[:0], None, 3)
    with pytest.raises(ValueError, match="max_children"):
        svr.DraftTree(z, None, 3, 2 ** 32 + 1)
    mask = torch.zeros((3, 1), dtype=torch.int64)
    with pytest.raises(ValueError, match="mask or positions"):
        svr.moe_tree_plan(tree, z[:1], None, None)
    with pytest.raises(ValueError, match="mask: expected torch.int64"):
        svr.moe_tree_plan(tree, z[:1], mask.int(), None)
    with pytest.raises(ValueError, match="positions: expected shape"):
        svr.moe_tree_plan(tree, z[:1], mask, z[:2])
    with pytest.raises(ValueError, match="seq_lens: expected shape"):
        svr.moe_tree_plan(tree, z, mask, z)
    with pytest.raises(ValueError, match="parents: expected 4 rows"):
        svr.moe_tree_plan(tree, z[:1], torch.zeros((4, 1), dtype=torch.int64), None)
    with pytest.raises(ValueError, match="device tensor"):
        svr.moe_tree_plan(tree, z[:1], mask, z)

    x, f = torch.zeros((3, 10)), torch.zeros(3)
    out = dict(accepted=torch.zeros((1, 3), **i32), n_accepted=z[:1], ws=torch.zeros(8, dtype=torch.uint8))
    call = lambda *a, **kw: svr.moe_verify_sample(tree, *a, **{**out, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="vocabulary"):
        call(x[0], z, f, f[:1])
    with pytest.raises(ValueError, match="whole rows"):
        call(torch.zeros((10, 3)).T, z, f, f[:1])
    with pytest.raises(ValueError, match="tokens: expected torch.int32"):
        call(x, z.long(), f, f[:1])
    with pytest.raises(ValueError, match="accept_u: expected torch.float32"):
        call(x, z, f.double(), f[:1])
    with pytest.raises(ValueError, match="sample_u: expected shape"):
        call(x, z, f, f)
    with pytest.raises(ValueError, match="draft_probs: expected float32"):
        call(x, z, f, f[:1], draft_probs=x.half())
    with pytest.raises(ValueError, match="accepted: expected shape"):
        call(x, z, f, f[:1], accepted=torch.zeros((1, 4), **i32))
    with pytest.raises(ValueError, match="pending_h: expected shape"):
        call(x, z, f, f[:1], verify_h=torch.zeros((3, 8)), pending_h=torch.zeros((1, 4)))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        call(x.double(), z, f, f[:1])
    with pytest.raises(ValueError, match="device tensor"):
        call(x, z, f, f[:1])

    d = svr.KvDesc(8, 2, 128, 16)
    batch = svr.KvBatch(torch.tensor([0, 3], **i32), z[:1], torch.zeros((1, 4), **i32), 3)
    cache = torch.zeros((4, 2, d.page_bytes), dtype=torch.uint8)
    q = torch.zeros((3, 8, 128))
    with pytest.raises(ValueError, match="mask: expected"):
        svr.moe_kv_tree_attention(d, batch, mask[:, 0], q, cache, q, ws=cache.view(-1))
    with pytest.raises(ValueError, match="mask: expected torch.int64"):
        svr.moe_kv_tree_attention(d, batch, mask.int(), q, cache, q, ws=cache.view(-1))
    with pytest.raises(ValueError, match="device tensor"):
        svr.moe_kv_tree_attention(d, batch, mask, q, cache, q, ws=cache.view(-1))
    path = torch.zeros((1, 3), **i32)
    with pytest.raises(ValueError, match="a cache is needed"):
        svr.moe_kv_commit(d, batch, path, z[:1], [])
    with pytest.raises(ValueError, match="twice"):
        svr.moe_kv_commit(d, batch, path, z[:1], [cache, cache])
    with pytest.raises(ValueError, match="one shape"):
        svr.moe_kv_commit(d, batch, path, z[:1], [cache, torch.zeros((5, 2, d.page_bytes), dtype=torch.uint8)])
    with pytest.raises(ValueError, match="path: expected shape"):
        svr.moe_kv_commit(d, batch, torch.zeros((2, 3), **i32), z[:1], [cache])
    with pytest.raises(ValueError, match="kept_lens is seq_lens"):
        svr.moe_kv_commit(d, batch, path, z[:1], [cache], batch.seq_lens)
    with pytest.raises(ValueError, match="or n_accepted"):
        svr.moe_kv_commit(d, batch, path, z[1:2], [cache], z[1:2])
    with pytest.raises(ValueError, match="device tensor"):
        svr.moe_kv_commit(d, batch, path, z[:1], [cache])


def test_the_binding_refuses_a_tree_on_another_device():
    z = torch.zeros(2, dtype=torch.int32)
    tree = svr.DraftTree(z, None, 2)
    m = dict(device="meta")
    i, f = torch.empty(1, dtype=torch.int32, **m), torch.empty(1, **m)
    with pytest.raises(ValueError, match="tree: expected tensors on meta"):
        svr.moe_tree_plan(tree, i, torch.empty((1, 1), dtype=torch.int64, **m), None)
    with pytest.raises(ValueError, match="tree: expected tensors on meta"):
        svr.moe_verify_sample(tree, torch.empty((1, 9), **m), i, f, f, torch.empty((1, 2), dtype=torch.int32, **m), i,
                              ws=torch.empty(0, dtype=torch.uint8, **m))


def test_random_trees_are_trees():
    rng = np.random.default_rng(0)
    for rows, kids in ((1, 1), (5, 1), (40, 2), (64, 9)):
        p = random_parents(rows, kids, rng)
        assert p[0] == -1 and all(0 <= x < j for j, x in enumerate(p) if j)
        assert max([p.count(i) for i in range(rows)]) <= kids
    off, par = forest([3, 0, 5], 2, rng)
    assert off.tolist() == [0, 3, 3, 8] and len(par) == 8


@pytest.mark.parametrize("heads,kv_heads,dim,rows", [(64, 4, 192, 4), (64, 4, 192, 15), (16, 2, 128, 61), (32, 8, 64, 4)])
def test_few_rows_need_the_workspace_of_what_runs_at_once(heads, kv_heads, dim, rows):
    """Row tiles of which eight or more run at once are cut into what does, with masks or without: 256
    compute units of two to four workgroups, whose rows are 16 or 32, D sums of 32 bits and two more."""
    off, table = torch.zeros(2, dtype=torch.int32), torch.zeros((1, 1000), dtype=torch.int32)
    n = svr.moe_kv_attention_workspace_bytes(svr.KvDesc(heads, kv_heads, dim, 64), svr.KvBatch(off, off[:1], table, rows), rows)
    most = 0
    for wide in (16, 32):
        for terms in (1, 2, 3):
            regs = wide // 16 * (dim // 8 * terms + dim // 4)  # of queries and sums
            groups = 4 if regs <= 48 else 3 if regs <= 72 else 2 if regs <= 160 else 1
            if wide == 16 or (rows * heads // kv_heads > 16 and groups >= 2):
                most = max(most, 256 * groups // kv_heads * kv_heads * wide)
    assert n <= most * (4 * dim + 8) + B.KV_COUNTER_BYTES + 255


def test_a_tree_without_a_number_of_children_leaves_none_out():
    i32 = dict(dtype=torch.int32)
    off, parents = torch.tensor([0, 9], **i32), torch.tensor([-1] + [0] * 8, **i32)
    for tree, kids in ((svr.DraftTree(off, parents, 9), 8), (svr.DraftTree(off, None, 9), 1),
                       (svr.DraftTree(off, parents, 1), 1), (svr.DraftTree(off, parents, 9, 2), 2),
                       (svr.DraftTree(off, parents, svr.TREE_MAX_ROWS), svr.TREE_MAX_ROWS - 1)):
        assert tree.max_children == tree.c(9).max_children == kids
        assert svr.moe_sample_workspace_bytes(tree, 9, 1000) > 0
