"""The paged 4-bit cache (include/moe_kv.h) on the GPU against the float64
oracle (oracle/kv_oracle.py), every call through the C ABI.

Append: the whole cache has to be equal byte for byte (keys are rounded from
64 bits, so a code next to a border falls on its own side), bytes of other
tokens unchanged.  Attention: everything that no row may see (free pages,
the rest of a last page, table entries without a token) holds NaN scales or
points nowhere; tolerances are derived in kv_support.attention_tolerance.
"""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev, log
from kv_support import TYPES, Plan, attention_tolerance, desc_of, rounded
from oracle import kv_oracle as ko

pytestmark = pytest.mark.gpu


def run_append(lay, plan, cache, q, k, v, **kw):
    """moe_kv_append on a copy of `cache`; returns it and q_out as float64."""
    c = dev(cache)
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    svr.moe_kv_append(desc_of(lay), plan.batch(), q, k, v, c, out, **kw)
    torch.cuda.synchronize()
    return c.cpu().numpy(), out.double().cpu().numpy()


def check_append(lay, plan, dtype, rng, norm=True, view=None, positions=None, scale=1.0):
    T, D = plan.T, lay.dim
    x = rng.standard_normal((T, lay.heads + 2 * lay.kv_heads, D)) * scale
    t, x64 = rounded(x, dtype)
    if view:
        t = view(t)
    hq, hk = lay.heads, lay.kv_heads
    w = [(1 + 0.1 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in "qk"]
    f = (10000.0 ** (-np.arange(0, lay.rotary, 2) / max(lay.rotary, 1))).astype(np.float32)
    cache = rng.integers(0, 256, plan.empty_cache().shape).astype(np.uint8)
    up = lambda a: None if a is None else dev(a)  # noqa: E731
    got, q_out = run_append(lay, plan, cache, t[:, :hq], t[:, hq:hq + hk], t[:, hq + hk:],
                            q_norm=up(w[0]), k_norm=up(w[1]), inv_freq=up(f) if lay.rotary else None,
                            positions=up(positions))
    want = cache.copy()
    ref = ko.append(lay, want, plan.offsets, plan.lens, plan.table, x64[:, :hq], x64[:, hq:hq + hk],
                    x64[:, hq + hk:], *w, f, positions)
    assert np.array_equal(got, want)
    n = plan.offsets[-1]
    # Norm: D + 4 roundings of the sum and the root, halved by it, then two
    # products; rotation: two products of sine and cosine (each rounded) and a
    # sum, of values up to |a| + |b|; then the type's own rounding.
    big = np.max(np.abs(ref[:n]), axis=-1, keepdims=True)
    tol = (D / 2 + 10) * 2.0 ** -24 * 2 * big + torch.finfo(TYPES[dtype]).eps / 2 * np.abs(ref[:n]) + 2.0 ** -25
    assert np.all(np.abs(q_out[:n] - ref[:n]) <= tol)
    assert np.all(np.isnan(q_out[n:]))  # rows behind the last sequence stay as they were


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,heads,kv_heads,page,rotary,interleaved", [
    (64, 3, 1, 16, 64, False), (128, 8, 8, 32, 32, True), (192, 16, 1, 64, 64, False),
    (192, 10, 2, 16, 192, True), (256, 5, 5, 128, 0, False), (256, 4, 2, 1024, 256, False),
    (64, 17, 1, 16, 16, False),
])
def test_append_bytes(dtype, dim, heads, kv_heads, page, rotary, interleaved):
    log(f"append {dtype} D={dim} {heads}/{kv_heads} page={page} rot={rotary}")
    rng = np.random.default_rng(dim + heads)
    lay = ko.Layout(heads, kv_heads, dim, page, 0, rotary, interleaved)
    plan = Plan(lay, [3, 0, 1, 5], [3, 7, page + 1, 2 * page + 2], rng, pad_rows=2)
    check_append(lay, plan, dtype, rng, norm=rotary != 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_rows_apart_and_unaligned(dtype):
    rng = np.random.default_rng(5)
    lay = ko.Layout(4, 2, 64, 16, 0, 32)
    plan = Plan(lay, [2, 3], [20, 33], rng)

    def apart(by, at):
        def f(t):
            buf = torch.zeros((t.shape[0], t[0].numel() + by + at), dtype=t.dtype, device="cuda")
            r = buf[:, at:at + t[0].numel()]
            r.copy_(t.flatten(1))
            return r.unflatten(1, t.shape[1:])
        return f
    check_append(lay, plan, dtype, rng, view=apart(64, 0))
    check_append(lay, plan, dtype, rng, view=apart(3, 0))   # rows at odd offsets
    check_append(lay, plan, dtype, rng, view=apart(8, 1))   # one element past an aligned start


def test_append_far_positions():
    rng = np.random.default_rng(6)
    lay = ko.Layout(2, 1, 128, 64, 0, 128)
    plan = Plan(lay, [4], [70], rng)
    pos = np.array([2 ** 30 + 7, 0, 999_983, -5], dtype=np.int32)
    check_append(lay, plan, "f32", rng, positions=pos)


def test_append_borders_of_the_codes():
    """Values on every midpoint of the grid, for blocks of every exponent that a type reaches."""
    lay = ko.Layout(1, 1, 64, 16)
    mid = np.array([0, 0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 6.5, 7, -0.25, -0.75, -5, -7, -0.0])
    exps = [0, 1, -1, 30, 100, 124, 125, -100, -126, -130, -140]
    rows = []
    for e in exps:
        for top in (7.0, 7.0000005, 6.0, 4.0):
            b = np.resize(mid, 31)
            rows.append(np.concatenate([[top], np.clip(b, -top, top)]) * 2.0 ** e)
    rows += [np.zeros(32), np.full(32, 3.4028234e38), np.full(32, 1e-45)]
    if len(rows) % 2:
        rows.append(np.ones(32))
    v = np.array(rows, dtype=np.float32).reshape(-1, 1, 64)
    T = len(v)
    plan = Plan(lay, [T], [T], np.random.default_rng(0))
    cache = plan.empty_cache()
    got, _ = run_append(lay, plan, cache, dev(v), dev(v), dev(v))
    want = cache.copy()
    ko.append(lay, want, plan.offsets, plan.lens, plan.table, v, v, v)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_a_token_that_is_not_finite_is_nan_for_those_who_see_it(where, what):
    rng = np.random.default_rng(7)
    lay = ko.Layout(4, 2, 64, 16, 0, 32)
    plan = Plan(lay, [4], [20], rng)
    q, q64 = rounded(rng.standard_normal((4, 4, 64)), "bf16")
    kv = {n: rng.standard_normal((4, 2, 64)) for n in "kv"}
    kv[where][2, 1, 40] = what  # the third row, the second head
    k, k64 = rounded(kv["k"], "bf16")
    v, v64 = rounded(kv["v"], "bf16")
    f = np.full(16, 0.5, np.float32)
    cache = plan.filled_cache(rng)
    got, _ = run_append(lay, plan, cache, q, k, v, inv_freq=dev(f))
    ko.append(lay, cache, plan.offsets, plan.lens, plan.table, q64, k64, v64, inv_freq=f)
    assert np.array_equal(got, cache)
    out = torch.empty_like(q)
    svr.moe_kv_attention(desc_of(lay), plan.batch(), q, dev(got), out)
    bad = torch.isnan(out).cpu().numpy()
    assert bad[2:, 2:].all() and not bad[:2].any() and not bad[:, :2].any()


def test_append_where_there_is_no_place():
    """Negative places, places beyond the table, pages outside the cache: queries are made, nothing is stored."""
    rng = np.random.default_rng(8)
    lay = ko.Layout(2, 1, 64, 16, 0, 32)
    plan = Plan(lay, [4, 3, 2], [2, 35, 18], rng, width=2)  # sequence 0: two rows before place 0; 1: beyond 32
    plan.table[2, 1] = plan.n_pages                        # sequence 2: its second page is not there
    check_append(lay, plan, "f32", rng)


def test_append_without_queries_and_read():
    rng = np.random.default_rng(9)
    lay = ko.Layout(6, 3, 192, 32)
    plan = Plan(lay, [3, 0, 2], [40, 5, 2], rng, pad_rows=1)
    plan.table[0, 1] = -1  # the page of sequence 0's rows (places 37 to 39)
    k, k64 = rounded(rng.standard_normal((6, 3, 192)), "f16")
    v, v64 = rounded(rng.standard_normal((6, 3, 192)), "f16")
    v[3, 1, 7] = float("nan")
    v64[3, 1, 7] = np.nan
    c = dev(plan.empty_cache())
    svr.moe_kv_append(desc_of(lay), plan.batch(), None, k, v, c, None)
    want = plan.empty_cache()
    ko.append(lay, want, plan.offsets, plan.lens, plan.table, np.zeros((6, 6, 192)), k64, v64)
    assert np.array_equal(c.cpu().numpy(), want)
    ko_, vo = (torch.full((6, 3, 192), 7.0, device="cuda") for _ in "kv")
    svr.moe_kv_read(desc_of(lay), plan.batch(), c, ko_, vo)
    ko_, vo = ko_.cpu().numpy(), vo.cpu().numpy()
    for h in range(3):
        K, V, _ = ko.stored(lay, want, plan.table[2], 2, h)
        assert np.array_equal(ko_[3:5, h], K, equal_nan=True) and np.array_equal(vo[3:5, h], V)
    assert np.isnan(ko_[3, 1]).all() and not vo[3, 1].any()
    assert not ko_[:3].any() and not vo[:3].any()   # not stored: zeros
    assert (ko_[5] == 7).all() and (vo[5] == 7).all()  # no sequence: left alone
    only = torch.empty((6, 3, 192), device="cuda")
    svr.moe_kv_read(desc_of(lay), plan.batch(), c, None, only)
    assert np.array_equal(only[:5].cpu().numpy(), vo[:5])


def check_attention(lay, plan, cache, dtype, rng, scale=None, q=None, want_lse=True, ws=None):
    T = plan.T
    qt, q64 = rounded(rng.standard_normal((T, lay.heads, lay.dim)), dtype) if q is None else q
    out = torch.full((T, lay.heads, lay.dim), 77.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.full((T, lay.heads), 77.0, device="cuda") if want_lse else None
    svr.moe_kv_attention(desc_of(lay, scale or 0.0), plan.batch(), qt, dev(cache), out, lse, ws=ws)
    torch.cuda.synchronize()
    ref, rl, size, reach, seen = ko.attention(lay, cache, plan.offsets, plan.lens, plan.table, q64, scale)
    n = plan.offsets[-1]
    got = out.double().cpu().numpy()
    assert (got[n:] == 77).all()
    tol = attention_tolerance(dtype, ref, size, reach, seen, lay.dim)[:n]
    err = np.abs(got[:n] - ref[:n])
    assert np.all(err <= tol), (np.nanmax(err - tol), np.nanmax(err))
    if want_lse:
        g = lse.double().cpu().numpy()
        assert (g[n:] == 77).all()
        g, r = g[:n], rl[:n]
        empty = np.isneginf(r)
        assert np.array_equal(np.isneginf(g), empty)
        # The score's roundings, the weights' sum (a rounding for each token), the logarithm and its sum.
        u = 2.0 ** -24
        t = (lay.dim + 4) * u * reach[:n] + (64 + seen[:n, None]) * u + 8 * u * np.abs(np.where(empty, 0, r))
        assert np.all(np.abs(g[~empty] - r[~empty]) <= t[~empty])
    return got, ref


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,heads,kv_heads,page,window", [
    (64, 4, 4, 16, 0), (128, 8, 2, 32, 0), (192, 16, 1, 64, 0), (256, 10, 2, 16, 0),
    (192, 32, 2, 16, 7), (128, 5, 1, 64, 100), (64, 64, 1, 128, 33), (256, 16, 1, 32, 64),
])
def test_attention_batches(dtype, dim, heads, kv_heads, page, window):
    log(f"attention {dtype} D={dim} {heads}/{kv_heads} page={page} W={window}")
    rng = np.random.default_rng(dim * heads + page)
    lay = ko.Layout(heads, kv_heads, dim, page, window)
    # Lengths of one token, a page, odd ones; no row; a length of zero; fewer tokens than rows.
    plan = Plan(lay, [1, 4, 0, 3, 2, 5, 1], [1, 4, 9, 130, 257, 3, 0], rng, pad_rows=3)
    got, _ = check_attention(lay, plan, plan.filled_cache(rng), dtype, rng)
    i = plan.offsets[5]
    assert not got[i:i + 2].any()             # two rows before place 0 see nothing
    assert not got[plan.offsets[6]].any()     # an empty sequence


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 33])
def test_attention_rows_share_a_tile(rows):
    rng = np.random.default_rng(rows)
    for heads, kv_heads in ((16, 1), (6, 2)):
        lay = ko.Layout(heads, kv_heads, 64, 16)
        plan = Plan(lay, [rows, 1], [rows + 61, 200], rng)
        check_attention(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("dtype,dim", [("bf16", 192), ("f32", 64), ("f16", 128)])
def test_attention_over_many_tokens(dtype, dim):
    """Long enough for every split of the axis; a table wider than the tokens."""
    rng = np.random.default_rng(11)
    lay = ko.Layout(8, 1, dim, 64)
    plan = Plan(lay, [4], [3001], rng, width=200)
    check_attention(lay, plan, plan.filled_cache(rng), dtype, rng)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f32", 64), ("f16", 64), ("bf16", 128), ("f16", 128),
                                       ("f32", 128), ("bf16", 192), ("f16", 192), ("f32", 192)])
@pytest.mark.parametrize("lens", [[2900], [1800, 333]])
def test_attention_of_a_verify_batch_in_a_long_table(dtype, dim, lens):
    """Tables that room for any length makes long: parts by the largest workgroups, most of them not in use."""
    log(f"long table {dtype} D={dim} {lens}")
    rng = np.random.default_rng(dim + len(lens))
    lay = ko.Layout(10, 1, dim, 64)
    plan = Plan(lay, [4] * len(lens), lens, rng, width=700)
    check_attention(lay, plan, plan.filled_cache(rng), dtype, rng)


def test_attention_calls_of_all_kinds_on_one_workspace():
    """Parts joined by the last workgroup or by a second kernel, in turn: every call leaves the counters zero."""
    rng = np.random.default_rng(54)
    cases = []
    for lay, rows, lens, dtype, width in (
            (ko.Layout(8, 1, 192, 16), [1], [900], "bf16", None), (ko.Layout(8, 2, 64, 16), [4, 2], [700, 90], "f32", 400),
            (ko.Layout(16, 2, 128, 32), [2] * 30, list(range(2, 32 * 40, 42))[:30], "f16", None),
            (ko.Layout(32, 2, 64, 16), [4], [600], "bf16", 3000)):
        plan = Plan(lay, rows, lens, rng, width=width)
        q, _ = rounded(rng.standard_normal((plan.T, lay.heads, lay.dim)), dtype)
        cases.append((desc_of(lay), plan.batch(), q, dev(plan.filled_cache(rng))))
    n = [svr.moe_kv_attention_workspace_bytes(d, b, len(q)) for d, b, q, _ in cases]
    assert all(n)
    ws = torch.full((max(n),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:16384].zero_()
    want = []
    for d, b, q, c in cases:
        out = torch.empty_like(q)
        svr.moe_kv_attention(d, b, q, c, out)
        want.append(out)
    for i in (0, 1, 2, 3, 2, 0, 0, 3, 1, 2):
        d, b, q, c = cases[i]
        out = torch.full_like(q, float("nan"))
        svr.moe_kv_attention(d, b, q, c, out, ws=ws)
        assert torch.equal(out, want[i]), i
        assert not ws[:16384].any(), i


@pytest.mark.parametrize("seqs,heads,kv_heads,page,window", [(2, 8, 2, 16, 0), (64, 4, 2, 32, 0), (65, 6, 3, 16, 0),
                                                             (150, 2, 1, 16, 0), (70, 3, 1, 16, 120)])
def test_attention_over_uneven_sequences(seqs, heads, kv_heads, page, window):
    """One long sequence among short and empty ones: the splits of a batch are shared out by its lengths,
    a wave at a time (of 64 sequences)."""
    log(f"uneven {seqs} {heads}/{kv_heads} W={window}")
    rng = np.random.default_rng(seqs)
    lay = ko.Layout(heads, kv_heads, 64, page, window)
    rows = rng.integers(0, 4, seqs)
    lens = rows + rng.integers(0, 90, seqs)
    rows[seqs // 2], lens[seqs // 2] = 41, 2100
    rows[-1], lens[-1] = 2, 700
    plan = Plan(lay, list(rows), list(lens), rng, pad_rows=1)
    check_attention(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("seqs,kv_heads,rows", [(40, 8, 20), (1100, 2, 9)])
def test_attention_over_many_sequences_of_several_row_tiles(seqs, kv_heads, rows):
    """Rows of uneven counts, one sequence of the most, with no split; too many sequences to look up."""
    log(f"row tiles {seqs}")
    rng = np.random.default_rng(seqs)
    lay = ko.Layout(4 * kv_heads, kv_heads, 64, 16)
    r = rng.integers(0, 4, seqs)
    r[seqs // 3], r[-1] = rows, rows - 1
    plan = Plan(lay, list(r), list(r + rng.integers(0, 30, seqs)), rng, pad_rows=1)
    check_attention(lay, plan, plan.filled_cache(rng), "bf16", rng)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_a_padded_batch(dtype):
    """Many rows of no sequence: the workspace is that of the sequences' rows."""
    rng = np.random.default_rng(51)
    lay = ko.Layout(8, 2, 64, 16)
    plan = Plan(lay, [3, 1], [1500, 700], rng, pad_rows=200)
    check_attention(lay, plan, plan.filled_cache(rng), dtype, rng)
    d = desc_of(lay)
    assert svr.moe_kv_attention_workspace_bytes(d, plan.batch(), 204) == \
        svr.moe_kv_attention_workspace_bytes(d, plan.batch(), 3000)


def test_attention_window_as_large_as_its_type():
    rng = np.random.default_rng(52)
    for window in (2 ** 31 - 1, 2 ** 30, 2 ** 20):
        lay = ko.Layout(4, 2, 64, 16, window)
        plan = Plan(lay, [6, 2], [3, 100], rng)  # three rows before place 0
        check_attention(lay, plan, plan.filled_cache(rng), "f32", rng)


def test_attention_makes_its_workspace_on_the_stream_of_the_call():
    rng = np.random.default_rng(53)
    lay = ko.Layout(8, 1, 64, 16)
    plan = Plan(lay, [4], [2000], rng)
    q, _ = rounded(rng.standard_normal((4, 8, 64)), "bf16")
    d, batch, cache = desc_of(lay), plan.batch(), dev(plan.filled_cache(rng))
    want = torch.empty_like(q)
    svr.moe_kv_attention(d, batch, q, cache, want)
    torch.cuda.synchronize()
    side, n = torch.cuda.Stream(), svr.moe_kv_attention_workspace_bytes(d, batch, 4)
    assert n > 0
    outs = []
    for _ in range(20):
        out = torch.empty_like(q)
        svr.moe_kv_attention(d, batch, q, cache, out, stream=side)
        outs.append(out)
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)  # what this stream may be given
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_attention_where_one_score_stands_out():
    """Peaked rows, and maxima that keep growing along the axis (every tile rescales)."""
    rng = np.random.default_rng(12)
    lay = ko.Layout(4, 1, 64, 16)
    plan = Plan(lay, [2], [1500], rng)
    cache = plan.filled_cache(rng)
    for t in range(1500):
        page, o = ko.slot(lay, plan.table[0], plan.n_pages, t)
        kc, _, ks, _ = ko.page_parts(lay, cache[page, 0])
        kc[o], ks[o] = 0x22, 110 + t // 100  # all channels alike, growing
    q = np.zeros((2, 4, 64))
    q[:, 0], q[:, 1], q[:, 2], q[:, 3] = 40.0, 3.0, -40.0, rng.standard_normal(64)
    check_attention(lay, plan, cache, "f32", rng, q=rounded(q, "f32"))
    check_attention(lay, plan, cache, "bf16", rng, q=rounded(q, "bf16"), scale=0.01)


def test_attention_hides_pages_that_are_not_there():
    rng = np.random.default_rng(13)
    lay = ko.Layout(4, 2, 128, 16)
    plan = Plan(lay, [3, 2], [100, 40], rng)
    cache = plan.filled_cache(rng)
    plan.table[0, 2], plan.table[0, 5], plan.table[1, 0] = -1, plan.n_pages, 2 ** 31 - 1
    cache[0] = 0xFF  # whatever stands in a page that a hidden token could be read from
    for b in range(2):
        plan.table[b][plan.table[b] == 0] = -7
    check_attention(lay, plan, cache, "bf16", rng)
    plan.table[:] = -1
    got, _ = check_attention(lay, plan, cache, "f32", rng)
    assert not got[:plan.offsets[-1]].any()


def test_attention_lengths_beyond_the_table():
    rng = np.random.default_rng(14)
    lay = ko.Layout(2, 1, 64, 16)
    plan = Plan(lay, [2, 2], [30, 64], rng, width=2)
    check_attention(lay, plan, plan.filled_cache(rng), "f32", rng)


def test_attention_leaves_rows_beyond_max_rows():
    rng = np.random.default_rng(15)
    lay = ko.Layout(2, 1, 64, 16)
    plan = Plan(lay, [5, 2], [30, 20], rng)
    plan.max_rows = 3
    q, q64 = rounded(rng.standard_normal((7, 2, 64)), "bf16")
    cache = plan.filled_cache(rng)
    out = torch.full((7, 2, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    svr.moe_kv_attention(desc_of(lay), plan.batch(), q, dev(cache), out)
    ref, _, size, reach, seen = ko.attention(lay, cache, plan.offsets, plan.lens, plan.table, q64)
    got = out.double().cpu().numpy()
    assert (got[3:5] == 77).all()
    keep = [0, 1, 2, 5, 6]
    tol = attention_tolerance("bf16", ref, size, reach, seen, 64)
    assert np.all(np.abs(got - ref)[keep] <= tol[keep])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_queries_apart_and_unaligned(dtype):
    rng = np.random.default_rng(16)
    lay = ko.Layout(4, 2, 64, 16)
    plan = Plan(lay, [2, 3], [20, 33], rng)
    cache = plan.filled_cache(rng)
    t, q64 = rounded(rng.standard_normal((5, 4, 64)), dtype)
    for width, at in ((320, 32), (259, 0), (264, 1)):
        buf = torch.zeros((5, width), dtype=t.dtype, device="cuda")
        q = buf[:, at:at + 256]
        q.copy_(t.flatten(1))
        check_attention(lay, plan, cache, dtype, rng, q=(q.unflatten(1, (4, 64)), q64))


def test_cache_beyond_four_gibibytes():
    """The last pages of a cache of 4.6 GB: offsets that pass 32 bits."""
    rng = np.random.default_rng(17)
    lay = ko.Layout(8, 8, 256, 1024)
    plan = Plan(lay, [2], [40], rng, spare=0)
    n = 2100
    assert n * 8 * lay.page_bytes > 4.2 * 2 ** 30
    big = svr.kv_cache(desc_of(lay), n)
    small = plan.empty_cache(0)
    k, k64 = rounded(rng.standard_normal((2, 8, 256)), "bf16")
    v, v64 = rounded(rng.standard_normal((2, 8, 256)), "bf16")
    small[:] = plan.filled_cache(rng)
    big[n - 1] = dev(small[plan.table[0, 0]])
    batch = svr.KvBatch(dev(plan.offsets), dev(plan.lens), dev(np.array([[n - 1]], np.int32)), 2)
    q, q64 = rounded(rng.standard_normal((2, 8, 256)), "bf16")
    qo, out = torch.empty_like(q), torch.empty_like(q)
    svr.moe_kv_append(desc_of(lay), batch, q, k, v, big, qo)
    svr.moe_kv_attention(desc_of(lay), batch, qo, big, out)
    ko.append(lay, small, plan.offsets, plan.lens, plan.table, q64, k64, v64)
    assert np.array_equal(big[n - 1].cpu().numpy(), small[plan.table[0, 0]])
    assert torch.equal(qo, q)  # neither norm nor rotation
    ref, _, size, reach, seen = ko.attention(lay, small, plan.offsets, plan.lens, plan.table, q64)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= attention_tolerance("bf16", ref, size, reach, seen, 256))


def test_append_and_attention_replayed_from_a_graph():
    """Captured once, replayed with eager work between; another stream and another workspace meanwhile."""
    rng = np.random.default_rng(18)
    lay = ko.Layout(16, 2, 128, 16, 0, 64)
    plan = Plan(lay, [4, 4], [300, 41], rng)
    q, _ = rounded(rng.standard_normal((8, 16, 128)), "bf16")
    k, _ = rounded(rng.standard_normal((8, 2, 128)), "bf16")
    v, _ = rounded(rng.standard_normal((8, 2, 128)), "bf16")
    f = dev((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32))
    d, batch = desc_of(lay), plan.batch()
    cache = dev(plan.filled_cache(rng))
    start = cache.clone()
    qo, out = torch.empty_like(q), torch.empty_like(q)
    ws, ws2 = svr.kv_workspace(d, batch, 8), svr.kv_workspace(d, batch, 8)

    def step(c, qo, out, ws, stream=None):
        svr.moe_kv_append(d, batch, q, k, v, c, qo, inv_freq=f, stream=stream)
        svr.moe_kv_attention(d, batch, qo, c, out, ws=ws, stream=stream)

    step(cache, qo, out, ws)
    torch.cuda.synchronize()
    want, want_cache = out.clone(), cache.clone()
    g, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        step(cache, qo, out, ws)
    c2, qo2, out2 = start.clone(), torch.empty_like(q), torch.empty_like(q)
    for i in range(4):
        cache.copy_(start)
        out.fill_(float("nan"))
        out2.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        step(c2, qo2, out2, ws2, stream=other)  # two calls at once
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cache, want_cache), i
        assert torch.equal(out2, want) and torch.equal(c2, want_cache), i


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn, with eager calls on the same workspace between, at lengths that change."""
    rng = np.random.default_rng(55)
    lay = ko.Layout(8, 2, 128, 16)
    plan = Plan(lay, [2, 1, 3], [900, 200, 500], rng)
    d, batch, cache = desc_of(lay), plan.batch(), dev(plan.filled_cache(rng))
    one = svr.KvBatch(dev(np.array([0, 2], np.int32)), batch.seq_lens[:1].clone(), batch.page_table[:1].contiguous(), 2)
    q, _ = rounded(rng.standard_normal((6, 8, 128)), "f16")
    q1 = q[:2].clone()
    ws = torch.zeros(max(svr.moe_kv_attention_workspace_bytes(d, batch, 6),
                         svr.moe_kv_attention_workspace_bytes(d, one, 2)), dtype=torch.uint8, device="cuda")
    calls = ((batch, q, torch.empty_like(q)), (one, q1, torch.empty_like(q1)))
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for g, (b, x, out) in zip(graphs, calls):
        svr.moe_kv_attention(d, b, x, cache, out, ws=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            svr.moe_kv_attention(d, b, x, cache, out, ws=ws)
    for lens in ([900, 200, 500], [40, 200, 3], [899, 1, 77]):
        batch.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        one.seq_lens.fill_(lens[0])
        want = []
        for b, x, out in calls:
            svr.moe_kv_attention(d, b, x, cache, out)
            want.append(out.clone())
        for i in (0, 1, 1, 0, 0, 1):
            calls[i][2].fill_(float("nan"))
            graphs[i].replay()
            assert torch.equal(calls[i][2], want[i]), (lens, i)
            eager = torch.empty_like(calls[1 - i][2])
            svr.moe_kv_attention(d, calls[1 - i][0], calls[1 - i][1], cache, eager, ws=ws)
            assert torch.equal(eager, want[1 - i]), (lens, i)


def test_rejected_drafts_are_overwritten():
    """A verify round whose tail is rejected: lower lengths and append again gives the cache of a clean run."""
    rng = np.random.default_rng(19)
    lay = ko.Layout(8, 2, 64, 16)
    first = Plan(lay, [4], [35], rng)
    cache = first.filled_cache(rng)
    d = desc_of(lay)
    x = [rounded(rng.standard_normal((4, 2, 64)), "bf16")[0] for _ in range(4)]
    q, q64 = rounded(rng.standard_normal((4, 8, 64)), "bf16")
    c = dev(cache)
    svr.moe_kv_append(d, first.batch(), None, x[0], x[1], c, None)
    # One draft of three accepted: places 31 and 32 stay, the next round starts at 33.
    second = Plan(lay, [4], [37], rng)
    second.table, second.n_pages = first.table, first.n_pages
    svr.moe_kv_append(d, second.batch(), None, x[2], x[3], c, None)
    want = cache.copy()
    a = [t.double().cpu().numpy() for t in x]
    zq = np.zeros((2, 8, 64))
    ko.append(lay, want, [0, 2], [33], first.table, zq, a[0][:2], a[1][:2])
    ko.append(lay, want, [0, 4], [37], first.table, q64, a[2], a[3])
    assert np.array_equal(c.cpu().numpy(), want)
    check_attention(lay, second, want, "bf16", rng, q=(q, q64))


@pytest.mark.parametrize("dim,heads,kv_heads,rows,length,width", [
    (64, 8, 2, 1, 1500, None), (128, 16, 1, 4, 3001, None), (192, 16, 1, 4, 2500, 700), (256, 8, 1, 2, 1200, None),
    (192, 6, 1, 33, 900, None)])
def test_bf16_attention_adds_no_error_to_the_rounding_of_its_result(dim, heads, kv_heads, rows, length, width):
    """The error of a weight shrinks with the tokens as the result does, so what counts is its share: with 16
    bits at most 2^-16 of a weight, and about sqrt(dim) 2^-24 of the scores' sizes, which is below 2^-13 here, it is a
    32nd of the rounding's 2^-8, and a thousandth of the sum of squares.  5% are allowed; weights of 8 bits make 40%."""
    log(f"bf16 precision D={dim} {rows} rows over {length}")
    rng = np.random.default_rng(dim + rows)
    lay = ko.Layout(heads, kv_heads, dim, 32)
    plan = Plan(lay, [rows], [length], rng, width=width)
    cache = plan.filled_cache(rng)
    q, q64 = rounded(rng.standard_normal((rows, heads, dim)), "bf16")
    out = torch.empty_like(q)
    svr.moe_kv_attention(desc_of(lay), plan.batch(), q, dev(cache), out)
    ref, *_ = ko.attention(lay, cache, plan.offsets, plan.lens, plan.table, q64)
    rounding = torch.from_numpy(ref).bfloat16().double().numpy() - ref
    err = out.double().cpu().numpy() - ref
    share = np.sqrt(np.mean(err ** 2) / np.mean(rounding ** 2))
    log(f"  error over rounding {share:.4f}")
    assert share <= 1.05


def check_attention_of(lay, plan, cache, dtype, rng, picks, ws=None, q=None):
    """check_attention of a large batch, with the oracle on the sequences `picks` only."""
    q, q64 = rounded(rng.standard_normal((plan.T, lay.heads, lay.dim)), dtype) if q is None else q
    out = torch.full_like(q, 77.0)
    svr.moe_kv_attention(desc_of(lay), plan.batch(), q, dev(cache), out, ws=ws)
    got = out.double().cpu().numpy()
    assert (got[plan.offsets[-1]:] == 77).all() and not (got[:plan.offsets[-1]] == 77).any()
    for b in picks:
        first, end = int(plan.offsets[b]), int(plan.offsets[b + 1])
        pieces = [(first, end)]
        if end - first > 200:  # some rows of a prompt: as if they were the last ones
            pieces = [(i, i + 40) for i in (first, (first + end) // 2, end - 40)]
        for i, j in pieces:
            ref, _, size, reach, seen = ko.attention(lay, cache, [0, j - i], plan.lens[b:b + 1] - (end - j),
                                                     plan.table[b:b + 1], q64[i:j])
            err = np.abs(got[i:j] - ref)
            assert np.all(err <= attention_tolerance(dtype, ref, size, reach, seen, lay.dim)), (b, i, np.nanmax(err))
    return got[:plan.offsets[-1]]


@pytest.mark.parametrize("seqs,heads,kv_heads,rows", [(1100, 6, 3, 500), (1024, 8, 1, 700), (300, 10, 2, 900),
                                                      (5, 15, 3, 500)])
def test_attention_of_a_prompt_among_many_sequences(seqs, heads, kv_heads, rows):
    """More row tiles than lie side by side (64), of one sequence or two; heads that do not divide the dies."""
    log(f"prompt of {rows} rows among {seqs}, {heads}/{kv_heads}")
    rng = np.random.default_rng(seqs + rows)
    lay = ko.Layout(heads, kv_heads, 64, 16)
    r = rng.integers(0, 3, seqs)
    r[seqs // 2], r[-1] = rows, rows // 3
    plan = Plan(lay, list(r), list(r + rng.integers(0, 30, seqs)), rng, pad_rows=1)
    picks = [seqs // 2, seqs - 1, 0, 1] + list(rng.integers(0, seqs, 40))
    check_attention_of(lay, plan, plan.filled_cache(rng), "bf16", rng, picks)


def test_attention_of_a_prompt_among_thousands_of_sequences():
    """Row tiles of as many rows for every sequence would be more workgroups than a launch can have."""
    rng = np.random.default_rng(61)
    lay = ko.Layout(64, 4, 64, 16)
    seqs, rows = 4100, 2048
    assert seqs * (rows * 16 // 32) * 4 * 256 >= 2 ** 32
    r, lens = np.ones(seqs, int), 1 + rng.integers(0, 4, seqs)
    r[777], lens[777] = rows, rows + 20
    plan = Plan(lay, list(r), list(lens), rng)
    cache = rng.integers(0, 256, plan.empty_cache().shape).astype(np.uint8)
    cache[..., 16 * 64:] = 126  # scales
    check_attention_of(lay, plan, cache, "bf16", rng, [777, 0, 776, 778, seqs - 1] + list(rng.integers(0, seqs, 40)))


@pytest.mark.parametrize("dtype,seqs,heads,kv_heads,dim,window,rows,length", [
    ("bf16", 97, 8, 8, 64, 0, 1, 3000), ("f16", 300, 16, 4, 128, 0, 2, 4000), ("f32", 700, 8, 8, 64, 0, 1, 5000),
    ("bf16", 100, 20, 4, 64, 0, 150, 3000), ("bf16", 130, 16, 8, 192, 2500, 3, 4000), ("f16", 64, 16, 16, 64, 0, 1, 2000),
    ("bf16", 2, 16, 16, 64, 0, 1, 2000), ("f32", 66, 4, 4, 256, 0, 4, 2500), ("bf16", 4000, 2, 1, 64, 0, 1, 30000)])
def test_attention_of_a_long_sequence_among_many(dtype, seqs, heads, kv_heads, dim, window, rows, length):
    """More sequences than run at once, of which a few are cut: each finds its parts among those of the others,
    in a workspace that goes by neither their rows nor their number; again where none is long."""
    log(f"long among many {dtype} D={dim} {seqs} of {heads}/{kv_heads} W={window}")
    rng = np.random.default_rng(seqs + dim)
    lay = ko.Layout(heads, kv_heads, dim, 16, window)
    r = rng.integers(0, 3, seqs)
    lens = r + rng.integers(0, 30, seqs)
    long = sorted({0, seqs // 2, seqs - 1}) if seqs > 2 else [1]
    for n, b in enumerate(long):
        r[b], lens[b] = max(1, rows - n), length // (n + 1)
    plan = Plan(lay, list(r), list(lens), rng, pad_rows=2)
    cache = rng.integers(0, 256, plan.empty_cache().shape).astype(np.uint8)
    cache[..., 16 * dim:] = rng.integers(124, 128, cache[..., 16 * dim:].shape)  # scales
    n = svr.moe_kv_attention_workspace_bytes(desc_of(lay), plan.batch(), plan.T)
    assert 0 < n < 2 ** 26
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:16384].zero_()
    picks = sorted({*long, *rng.integers(0, seqs, 30).tolist()})
    q = rounded(rng.standard_normal((plan.T, heads, dim)), dtype)
    want = check_attention_of(lay, plan, cache, dtype, rng, picks, ws, q)
    assert not ws[:16384].any()
    full, plan.lens = plan.lens, np.minimum(plan.lens, 40).astype(np.int32)
    check_attention_of(lay, plan, cache, dtype, rng, picks, ws)
    plan.lens = full
    assert np.array_equal(check_attention_of(lay, plan, cache, dtype, rng, [], ws, q), want)
    assert not ws[:16384].any()


@pytest.mark.parametrize("dtype,dim,window,lens", [
    ("bf16", 256, 0, [2600]), ("f32", 256, 0, [2700, 400]), ("f16", 256, 0, [2600]), ("bf16", 192, 3000, [6000]),
    ("f16", 128, 2500, [5000, 4000]), ("f32", 64, 4000, [9000])])
def test_attention_of_parts_that_a_second_kernel_joins(dtype, dim, window, lens):
    """More than sixteen parts a row, at every head size, and of rows whose window begins inside the tokens."""
    log(f"second kernel {dtype} D={dim} W={window} {lens}")
    rng = np.random.default_rng(dim + window)
    lay = ko.Layout(4, 1, dim, 64, window)
    plan = Plan(lay, [2] * len(lens), lens, rng, width=300)
    check_attention(lay, plan, plan.filled_cache(rng), dtype, rng)


def test_attention_workspace_of_the_largest_batch_serves_the_others():
    """A server's prompt is not cut, its single sequences are: one workspace, made for the former."""
    rng = np.random.default_rng(62)
    lay = ko.Layout(16, 2, 128, 16)
    sizes = (([600, 1], [600, 300]), ([1], [2000]), ([4], [1500]), ([2] * 20, [90] * 20), ([1, 3], [2000, 40]),
             ([64], [900]), ([1], [3]))
    largest = svr.KvBatch(torch.zeros(21, dtype=torch.int32, device="cuda"),
                          torch.zeros(20, dtype=torch.int32, device="cuda"),
                          torch.zeros((20, 125), dtype=torch.int32, device="cuda"), 600)
    for dtype in TYPES:
        ws = svr.kv_workspace(desc_of(lay), largest, 601)
        for rows, lens in sizes:
            log(f"one workspace {dtype} {rows[:2]} {lens[:2]}")
            plan = Plan(lay, rows, lens, rng)
            check_attention_of(lay, plan, plan.filled_cache(rng), dtype, rng, sorted({0, len(rows) - 1}), ws)
            assert not ws[:16384].any()


@pytest.mark.parametrize("seqs", [62, 63, 64, 65, 127, 400, 4097])
def test_append_and_read_of_many_sequences(seqs):
    """On both sides of the lookup of a row's sequence by one load of all offsets, with empty sequences at
    either end; rows of no sequence hold NaN and stay out of the cache."""
    log(f"append of {seqs} sequences")
    rng = np.random.default_rng(seqs)
    lay = ko.Layout(2, 1, 64, 16, 0, 32)
    rows = rng.integers(0, 3, seqs)
    rows[0] = rows[-1] = 0
    rows[seqs // 2] = 5
    plan = Plan(lay, list(rows), list(rows + rng.integers(0, 20, seqs)), rng, pad_rows=3)
    n = int(plan.offsets[-1])
    x = rng.standard_normal((plan.T, 4, 64))
    x[n:] = np.nan
    t, x64 = rounded(x, "bf16")
    f = np.full(16, 0.25, np.float32)
    cache = rng.integers(0, 256, plan.empty_cache().shape).astype(np.uint8)
    got, q_out = run_append(lay, plan, cache, t[:, :2], t[:, 2:3], t[:, 3:], inv_freq=dev(f))
    want = cache.copy()
    ref = ko.append(lay, want, plan.offsets, plan.lens, plan.table, x64[:, :2], x64[:, 2:3], x64[:, 3:], inv_freq=f)
    assert np.array_equal(got, want)
    # A sine, a cosine, two products and a sum of 24 bits, of values up to |a| + |b|, then bf16's own rounding.
    tol = 10 * 2.0 ** -24 * np.max(np.abs(ref[:n]), -1, keepdims=True) * 2 + 2.0 ** -8 * np.abs(ref[:n])
    assert np.all(np.abs(q_out[:n] - ref[:n]) <= tol) and np.isnan(q_out[n:]).all()
    k, v = (torch.full((plan.T, 1, 64), 7.0, device="cuda") for _ in "kv")
    svr.moe_kv_read(desc_of(lay), plan.batch(), dev(want), k, v)
    k, v = k.cpu().numpy(), v.cpu().numpy()
    assert (k[n:] == 7).all() and (v[n:] == 7).all()
    for b in range(seqs):
        for i in range(plan.offsets[b], plan.offsets[b + 1]):
            page, o = ko.slot(lay, plan.table[b], plan.n_pages, int(plan.lens[b]) - int(plan.offsets[b + 1]) + i)
            kc, vc, ks, vs = ko.page_parts(lay, want[page, 0])
            assert np.array_equal(k[i, 0], ko.vector_values(kc[o], ks[o])), (b, i)
            assert np.array_equal(v[i, 0], ko.vector_values(vc[o], vs[o])), (b, i)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 192])
def test_append_norm_of_heads_of_any_size(dtype, dim):
    """Heads whose squares pass the range of 32 bits at either end, next to ordinary ones, without an epsilon."""
    log(f"norm of any size {dtype} D={dim}")
    rng = np.random.default_rng(dim)
    lay = ko.Layout(10, 2, dim, 16, 0, 32, eps=0.0)
    plan = Plan(lay, [5], [21], rng)
    scales = np.array([1, 1e-4, 1e3] if dtype == "f16" else [1e-43, 1e-30, 1e-20, 1e-15, 1, 1e15, 1e19, 1e25, 3e37])
    s = scales[(np.arange(5)[:, None] * 11 + np.arange(14)) % len(scales)]
    t, x64 = rounded(rng.uniform(0.5, 1, (5, 14, dim)) * rng.choice([-1, 1], (5, 14, dim)) * s[:, :, None], dtype)
    w = (1 + 0.1 * rng.standard_normal((2, dim))).astype(np.float32)
    f = np.full(16, 0.25, np.float32)
    cache = plan.empty_cache()
    got, q_out = run_append(lay, plan, cache, t[:, :10], t[:, 10:12], t[:, 12:], q_norm=dev(w[0]), k_norm=dev(w[1]),
                            inv_freq=dev(f))
    with np.errstate(invalid="ignore"):
        ref = ko.append(lay, cache, plan.offsets, plan.lens, plan.table, x64[:, :10], x64[:, 10:12], x64[:, 12:], *w, f)
    assert np.array_equal(got, cache)
    # As in check_append.
    big = np.max(np.abs(ref), axis=-1, keepdims=True)
    tol = (dim / 2 + 10) * 2.0 ** -24 * 2 * big + torch.finfo(TYPES[dtype]).eps / 2 * np.abs(ref) + 2.0 ** -25
    nothing = np.isnan(ref)  # bf16 has no 1e-43: heads of zeros, whose norm is 0 / 0
    assert nothing.any() == (dtype == "bf16") and np.array_equal(np.isnan(q_out), nothing)
    assert np.all((np.abs(q_out - ref) <= tol) | nothing)
