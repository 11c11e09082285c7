"""Sampled verification (include/moe_sample.h) on the GPU against the float64 oracle
(oracle/sample_oracle.py), every call through the C ABI.

Outputs are whole numbers and have to be equal.  They depend on comparisons of 64-bit numbers, which the
library and the oracle round differently: a weight is off by at most 8e-14 (its polynomial) and some 2^-53
for each of at most 30 operations, so a probability by twice that, 1.7e-13; a sum by 2^-53 for each of its
additions in a row, here at most 1500 times 2^-53 = 1.7e-13 (NumPy's pairwise and cumulative sums of rows
that weigh one; a tile's and its join's are fewer).  So no comparison whose sides lie 1e-12 apart (of a
probability of one) can fall differently; the oracle says how far apart the closest were, and every test
asserts that first."""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev, log
from kv_support import TYPES
from oracle import sample_oracle as so
from tree_support import forest, tree_of

pytestmark = pytest.mark.gpu

MARGIN = 1e-12


class Case:
    """Inputs of a call: logits and, for drawn drafts, probabilities close to theirs."""

    def __init__(self, rows, V, kids, rng, dtype="f32", drawn=False, masked=False, greedy=0.0, spread=3.0, pad=0,
                 near=0.4, max_rows=None, chain=None):
        self.offsets, self.parents = forest([int(r) for r in rows], kids, rng)
        if chain if chain is not None else kids == 1:
            self.parents = None
        T, B = int(self.offsets[-1]), len(rows)
        self.kids, self.V, self.pad, self.max_rows = kids, V, pad, max_rows or max(max(rows), 1)
        x = rng.standard_normal((T + pad, V)) * spread
        self.set_logits(x, dtype, masked, rng)
        y = np.where(np.isneginf(self.x), -np.inf, x + near * rng.standard_normal(x.shape))
        y = y - np.max(np.where(np.isneginf(y), -1e30, y), 1, keepdims=True)
        q = np.exp(y)
        self.q = (q / q.sum(1, keepdims=True)).astype(np.float32) if drawn else None
        self.tokens = np.zeros(T + pad, np.int32)
        up = np.arange(-1, T - 1) if self.parents is None else None
        for b in range(B):
            off = int(self.offsets[b])
            nth = {}
            for i in range(1, int(self.offsets[b + 1]) - off):
                p = off + (i - 1 if self.parents is None else int(self.parents[off + i]))
                nth[p] = nth.get(p, -1) + 1
                if drawn:
                    w = self.q[p].astype(np.float64)
                    self.tokens[off + i] = rng.choice(V, p=w / w.sum())
                else:
                    self.tokens[off + i] = np.argsort(-y[p], kind="stable")[min(nth[p], V - 1)]
        del up
        self.accept_u, self.sample_u = rng.random(T + pad).astype(np.float32), rng.random(B).astype(np.float32)
        self.temperature = (0.5 + rng.random(B)).astype(np.float32)
        self.temperature[rng.random(B) < greedy] = 0.0

    def set_logits(self, x, dtype, masked=False, rng=None):
        if masked:
            x = np.where(rng.random(x.shape) < 0.7, -np.inf, x)
        self.logits = torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype]).cuda()
        self.x = self.logits.double().cpu().numpy()

    def want(self):
        return so.verify(self.x, self.offsets, self.parents, self.tokens, self.accept_u, self.sample_u, self.max_rows,
                         self.kids, self.q, self.temperature)

    def tree(self):
        return tree_of(self.offsets, self.parents, self.max_rows, self.kids, self.pad)

    def device(self):
        """The call's tensors: (tree, logits, tokens, accept_u, sample_u), keywords."""
        return ((self.tree(), self.logits, dev(self.tokens), dev(self.accept_u), dev(self.sample_u)),
                dict(draft_probs=None if self.q is None else dev(self.q), temperature=dev(self.temperature)))

    def outputs(self):
        B = len(self.offsets) - 1
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.full((B, self.max_rows), -7, **i32), torch.full((B,), -7, **i32),
                torch.full((B, self.max_rows), -7, **i32))


def check(c, want=None, ws=None, margin=MARGIN, h=5, **kw):
    want = want or c.want()
    assert want["margin"] > margin, want["margin"]
    args, named = c.device()
    accepted, n, path = c.outputs()
    T, B = len(c.tokens), len(c.offsets) - 1
    vh = torch.randn((T, h), device="cuda")
    pending = torch.full((B, h), -7.0, device="cuda")
    svr.moe_verify_sample(*args, accepted, n, path, verify_h=vh, pending_h=pending, ws=ws, **{**named, **kw})
    torch.cuda.synchronize()
    got = dict(accepted=accepted.tolist(), path=path.tolist(), n_accepted=n.tolist())
    for b in range(B):
        if want["row"][b] is None:  # a sequence without rows: left as it was
            assert set(got["accepted"][b]) == set(got["path"][b]) == {-7} and got["n_accepted"][b] == -7
            assert (pending[b] == -7).all()
            continue
        for k in ("accepted", "path", "n_accepted"):
            assert got[k][b] == want[k][b], (k, b, got[k][b], want[k][b])
        assert torch.equal(pending[b], vh[want["row"][b]])
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("rows,V,kids", [
    ([4], 5000, 1), ([1], 1, 1), ([3, 1, 0, 5, 2], 1023, 1), ([7, 0, 12], 1024, 3), ([20], 1025, 2), ([9, 30, 2], 4097, 4),
    ([2] * 70, 300, 1), ([5, 6] * 20, 2049, 2),
])
def test_batches(dtype, drawn, rows, V, kids):
    log(f"sample {dtype} drawn={drawn} rows={rows[:5]} V={V} kids={kids}")
    rng = np.random.default_rng(V + kids + 10 * drawn)
    check(Case(rows, V, kids, rng, dtype, drawn, pad=3))


@pytest.mark.parametrize("drawn", [False, True])
def test_drafts_are_accepted_and_rejected(drawn):
    """Enough of both, at every length of the path."""
    rng = np.random.default_rng(50)
    c = Case([5] * 120, 400, 1, rng, drawn=drawn, near=0.5)
    got = check(c)
    assert set(got["n_accepted"]) == {0, 1, 2, 3, 4}
    c = Case([13] * 60, 300, 3, rng, drawn=drawn, near=0.8)
    got = check(c)
    assert len(set(got["n_accepted"])) >= 3
    # Second and third children too: a path through the first ones only would not tell them apart.
    want = c.want()
    firsts = sum(p[1] == 1 for p in want["path"])
    assert 0 < firsts < sum(p[1] > 0 for p in want["path"])


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("masked,greedy", [(True, 0.0), (True, 0.5), (False, 1.0)])
def test_masks_and_greedy_sequences(drawn, masked, greedy):
    rng = np.random.default_rng(51)
    check(Case([4, 9, 6, 1, 8], 2500, 2, rng, "bf16", drawn, masked, greedy))


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("temperature", [1e-45, 1e-30, 1e-6, 0.01, 100.0, 1e30, float("inf"), -1.0, float("nan"), -0.0])
def test_temperatures(drawn, temperature):
    """Up to one column's weight, and to all columns alike."""
    rng = np.random.default_rng(52)
    c = Case([5, 7], 1500, 2, rng, drawn=drawn)
    c.temperature[:] = temperature
    check(c)


def test_no_temperature_is_one():
    c = Case([5, 7], 1500, 2, np.random.default_rng(53))
    c.temperature[:] = 1.0
    check(c, temperature=None)


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("greedy", [0.0, 1.0])
def test_logits_that_are_not_finite(drawn, greedy):
    rng = np.random.default_rng(54)
    c = Case([3] * 8, 1100, 1, rng, drawn=drawn, greedy=greedy)
    x = c.x.copy()
    x[0] = -np.inf                       # no distribution: nothing accepted, no token
    x[3] = np.nan
    x[6, ::3] = np.nan                   # weight zero
    x[9, [5, 700, 1099]] = np.inf        # these three alike
    x[12, 1:] = -np.inf                  # one column
    x[15], x[15, 1024] = -np.inf, -3e38
    x[18, 7] = 3.4e38
    x[21, :1024] = -np.inf               # a tile of nothing
    c.logits, c.x = dev(x.astype(np.float32)), x.astype(np.float32).astype(np.float64)
    check(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("drawn", [False, True])
def test_masks_of_the_lowest_value_and_signalling_nan(dtype, drawn):
    rng = np.random.default_rng(70)
    c = Case([4] * 6, 1100, 1, rng, dtype, drawn)
    low = torch.finfo(TYPES[dtype]).min
    x = np.where(rng.random(c.x.shape) < 0.5, low, c.x)
    x[20:22] = low                      # a whole row: one weight for 16-bit types, none for float
    c.set_logits(x, dtype)
    bits = {"f32": (torch.int32, 0x7F800001), "bf16": (torch.int16, 0x7F81), "f16": (torch.int16, 0x7C01)}[dtype]
    c.logits.view(bits[0])[:, 5::7] = bits[1]   # NaN of the kind that an operation would trap on
    c.x = c.logits.double().cpu().numpy()
    assert np.isnan(c.x[:, 5::7]).all()
    check(c)
    c.temperature[:] = [np.inf, 1e30, 1e-30, 0.0, np.inf, 3e38]
    check(c)


def test_greedy_takes_the_lowest_of_equal_ones():
    c = Case([3, 3], 3000, 1, np.random.default_rng(55), "bf16", greedy=1.0)
    x = np.zeros((6, 3000))
    x[0, [2900, 1500, 17]] = 4.0
    x[1, [2048, 1023]] = 4.0
    c.set_logits(x, "bf16")
    c.tokens[:] = [0, 17, 1023, 0, 17, 5]
    got = check(c)
    assert got["accepted"] == [[17, 1023, 0], [0, -1, -1]]


@pytest.mark.parametrize("drawn", [False, True])
def test_the_same_token_twice_and_tokens_that_are_none(drawn):
    rng = np.random.default_rng(56)
    c = Case([6] * 40, 30, 5, rng, drawn=drawn)
    # Siblings: all children of the root.
    c.parents = np.tile(np.array([-1, 0, 0, 0, 0, 0], np.int32), 40)
    for b in range(40):
        c.tokens[6 * b + 1:6 * b + 6] = rng.choice([3, 7, -1, 30, 2 ** 31 - 1, 12], 5)
    c.accept_u[:] = 0.5 + 0.5 * c.accept_u
    check(c)
    # The same with tokens that have much of the weight.
    x = c.x.copy()
    x[:, [3, 7, 12]] += 8.0
    c.set_logits(x, "f32")
    got = check(c)
    assert 0 < sum(got["n_accepted"]) < 40


def test_children_from_max_children_on_are_never_accepted():
    rng = np.random.default_rng(57)
    for drawn in (False, True):
        c = Case([9] * 30, 50, 8, rng, drawn=drawn)
        c.parents = np.tile(np.array([-1] + [0] * 8, np.int32), 30)
        c.kids = 2
        got = check(c)
        assert max(max(p) for p in got["path"]) <= 2 < 8


def test_rows_that_are_no_nodes():
    """Rows from max_rows on, and parents that are not earlier rows."""
    rng = np.random.default_rng(58)
    for drawn in (False, True):
        c = Case([12, 9, 12], 200, 2, rng, drawn=drawn, max_rows=9)
        c.parents[[3, 14, 20]] = [3, -1, 2 ** 31 - 1]
        check(c)


def test_a_tree_of_one_parent_for_all():
    """More children than a wave has lanes."""
    rng = np.random.default_rng(59)
    for drawn, n in ((False, 300), (False, 65), (True, 4)):
        c = Case([n], 5000, n, rng, drawn=drawn, spread=1.0)
        c.parents = np.array([-1] + [0] * (n - 1), np.int32)
        if not drawn:
            c.tokens[:] = rng.permutation(5000)[:n]
            c.accept_u[:] = 1 - 2.0 ** -24  # all but certain to be rejected
        c.kids = n
        check(c)


@pytest.mark.parametrize("drawn", [False, True])
def test_random_numbers_at_their_ends(drawn):
    rng = np.random.default_rng(60)
    for u, s in ((0.0, 0.0), (1 - 2.0 ** -24, 1 - 2.0 ** -24), (0.0, 1 - 2.0 ** -24), (2.0 ** -24, 0.0)):
        c = Case([4, 6], 700, 2, rng, drawn=drawn)
        c.accept_u[:], c.sample_u[:] = u, s
        # (A number of 0 is the border of the first column, which both sides take alike: 0 < w.)
        check(c, margin=-1.0 if s == 0.0 or u == 0.0 else MARGIN)


def test_drafts_that_take_all_of_the_target():
    """Given drafts whose probabilities are nearly one: what is left is the rest, not a difference."""
    c = Case([2, 2, 2], 2000, 1, np.random.default_rng(61))
    x = np.full((6, 2000), -20.0)
    x[[0, 2, 4], [5, 1999, 1024]] = 0.0      # about 1 - 4e-6
    c.set_logits(x, "f32")
    c.tokens[[1, 3, 5]] = [5, 1999, 1024]
    c.temperature[:] = 1.0
    c.accept_u[:] = 1 - 2.0 ** -24
    got = check(c)
    assert got["n_accepted"] == [0, 0, 0]
    # Nothing left at all, by numbers that a caller should not give: the most likely token.
    x[:], x[[0, 2, 4], [5, 1999, 1024]] = -np.inf, 0.0
    c.set_logits(x, "f32")
    c.accept_u[:] = 1.0
    got = check(c, margin=-1.0)
    assert [a[0] for a in got["accepted"]] == [5, 1999, 1024]


def test_draft_probabilities_that_cover_the_target():
    """q above p everywhere (no distribution): nothing is left, the most likely token comes."""
    c = Case([2, 2], 1500, 1, np.random.default_rng(62), drawn=True)
    c.q[:] = 1.0
    c.accept_u[:] = 0.999
    got = check(c)
    assert [a[0] for a in got["accepted"]] == c.x[[0, 2]].argmax(1).tolist()
    c.q[0], c.q[2] = -1.0, np.nan  # as zero: every draft that has weight is accepted
    got = check(c)
    assert got["n_accepted"] == [1, 1]


def test_logits_and_probabilities_apart_and_unaligned():
    rng = np.random.default_rng(63)
    for dtype in ("f32", "bf16"):
        c = Case([4, 7], 1030, 2, rng, dtype, drawn=True)
        want = c.want()
        for width, at in ((1040, 8), (1033, 0), (1100, 1)):
            def apart(t):
                buf = torch.full((t.shape[0], width), float("nan"), dtype=t.dtype, device="cuda")
                r = buf[:, at:at + 1030]
                r.copy_(t)
                return r
            rows = c.logits
            c.logits = apart(rows)
            check(c, want, draft_probs=apart(dev(c.q)))
            c.logits = rows


@pytest.mark.parametrize("V", [131072, 262147])
@pytest.mark.parametrize("drawn", [False, True])
def test_large_vocabularies(V, drawn):
    rng = np.random.default_rng(64)
    check(Case([4, 9], V, 2, rng, "bf16", drawn, spread=2.0))


def test_a_vocabulary_of_several_passes():
    """More tiles than the last workgroup has threads."""
    rng = np.random.default_rng(65)
    V = 600_001
    for drawn in (False, True):
        check(Case([3], V, 1, rng, "f16", drawn, spread=1.0))


def test_many_rows_share_no_workgroup():
    rng = np.random.default_rng(66)
    check(Case([3] * 800, 3000, 1, rng, "bf16"))


def test_calls_of_all_kinds_on_one_workspace():
    rng = np.random.default_rng(67)
    cases = [Case([4], 9000, 1, rng), Case([9, 3, 0, 5], 700, 3, rng, "bf16", drawn=True), Case([2] * 50, 2100, 1, rng, "f16"),
             Case([6], 9000, 2, rng, drawn=True)]
    want = [c.want() for c in cases]
    n = max(svr.moe_sample_workspace_bytes(c.tree(), len(c.tokens), c.V) for c in cases)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:131072].zero_()
    for i in (0, 1, 2, 3, 1, 1, 0, 3, 2, 0):
        check(cases[i], want[i], ws=ws)
        assert not ws[:131072].any(), i


def test_two_streams_and_a_graph():
    """Two calls at once on workspaces of their own; captured calls that share one, replayed on new inputs."""
    rng = np.random.default_rng(68)
    cases = [Case([5, 6], 8000, 1, rng), Case([7, 4, 3], 6000, 2, rng, "bf16", drawn=True)]
    dev_in = [c.device() for c in cases]
    outs = [c.outputs() for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (a, kw), o, s in zip(dev_in, outs, streams):
            svr.moe_verify_sample(*a, *o, stream=s, **kw)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        w = c.want()
        assert w["margin"] > MARGIN
        assert o[0].tolist() == w["accepted"] and o[1].tolist() == w["n_accepted"] and o[2].tolist() == w["path"]

    big = max(cases, key=lambda c: svr.moe_sample_workspace_bytes(c.tree(), len(c.tokens), c.V))
    ws = svr.sample_workspace(big.tree(), len(big.tokens), big.V)
    side, graphs = torch.cuda.Stream(), []
    for (a, kw), o in zip(dev_in, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            svr.moe_verify_sample(*a, *o, ws=ws, **kw)
        graphs.append(g)
    for k in range(4):
        for c, (a, kw), o, g in zip(cases, dev_in, outs, graphs):
            c.accept_u, c.sample_u = (rng.random(len(x)).astype(np.float32) for x in (c.accept_u, c.sample_u))
            a[3].copy_(dev(c.accept_u))
            a[4].copy_(dev(c.sample_u))
            for t in o:
                t.fill_(-7)
            g.replay()
            torch.cuda.synchronize()
            w = c.want()
            assert w["margin"] > MARGIN
            assert o[0].tolist() == w["accepted"] and o[1].tolist() == w["n_accepted"] and o[2].tolist() == w["path"]
            assert not ws[:131072].any()


@pytest.mark.parametrize("kids,drawn", [(1, True), (3, True), (3, False)])
def test_tokens_are_distributed_as_the_targets(kids, drawn):
    """The first token of 16000 sequences of one pair of distributions, counted."""
    rng = np.random.default_rng(69)
    V, n, rows = 12, 16000 // (1 + kids) * 1, 1 + kids
    p = rng.dirichlet(np.ones(V))
    x = np.log(p).astype(np.float32)
    e = np.exp(x.astype(np.float64))
    p = e / e.sum()
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    offsets = np.arange(n + 1, dtype=np.int32) * rows
    parents = np.tile(np.array([-1] + [0] * kids, np.int32), n)
    if drawn:
        tokens = rng.choice(V, n * rows, p=q.astype(np.float64) / q.astype(np.float64).sum())
    else:
        tokens = np.tile(np.concatenate([[0], np.argsort(-q)[:kids]]), n)
    t = tree_of(offsets, parents, rows, kids)
    i32 = dict(dtype=torch.int32, device="cuda")
    accepted, count = torch.empty((n, rows), **i32), torch.empty(n, **i32)
    f = lambda m: dev(rng.random(m).astype(np.float32))  # noqa: E731
    svr.moe_verify_sample(t, dev(np.tile(x, (n * rows, 1))), dev(tokens.astype(np.int32)), f(n * rows), f(n), accepted,
                          count, draft_probs=dev(np.tile(q, (n * rows, 1))) if drawn else None)
    got = np.bincount(accepted[:, 0].cpu().numpy(), minlength=V)
    # Five standard deviations of each count.
    assert got.sum() == n and np.all(np.abs(got - n * p) <= 5 * np.sqrt(n * p * (1 - p)))
    assert 0 < int((count > 0).sum()) < n


@pytest.mark.parametrize("drawn", [False, True])
def test_rows_that_lie_beyond_32_bits(drawn):
    """Rows of logits and of probabilities so far apart that the last ones are more than 2^31 elements, and
    2^32 bytes, from the first."""
    c = Case([3], 1500, 1, np.random.default_rng(72), "bf16", drawn)
    want = c.want()

    def apart(t, stride):
        rows = torch.empty(2 * stride + 1500, dtype=t.dtype, device="cuda").as_strided((3, 1500), (stride, 1))
        rows.copy_(t)
        return rows

    c.logits = apart(c.logits, 2 ** 30 + 3)
    check(c, want, **(dict(draft_probs=apart(dev(c.q), 2 ** 30 + 1)) if drawn else {}))


def test_padded_batches_and_their_graph():
    """Rows behind the last sequence; a captured call replayed for other numbers of rows and sequences without any."""
    cases = [Case(rows, 2000, 2, np.random.default_rng(74 + i), "f32", drawn, pad=20 - sum(rows), max_rows=9,
                  chain=False)
             for i, rows in enumerate(([4, 9, 2], [1, 0, 0], [0, 8, 9], [5, 5, 5])) for drawn in (False, True)]
    for drawn in (False, True):
        first = next(c for c in cases if (c.q is not None) == drawn)
        args, named = first.device()
        args = (args[0], args[1].clone(), *args[2:])  # (the logits are the case's own)
        tree, q = args[0], named["draft_probs"]
        out = first.outputs()
        ws = svr.sample_workspace(tree, 20, 2000)
        call = lambda: svr.moe_verify_sample(*args, *out, **named, ws=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for c in [c for c in cases if (c.q is not None) == drawn] * 2:
            got = check(c, ws=ws)
            new, more = c.device()
            tree.q_offsets.copy_(new[0].q_offsets)
            tree.parents.copy_(new[0].parents)
            for a, b in zip(args[1:], new[1:]):
                a.copy_(b)
            named["temperature"].copy_(more["temperature"])
            if drawn:
                q.copy_(more["draft_probs"])
            for t in out:
                t.fill_(-7)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert [t.tolist() for t in out] == [got["accepted"], got["n_accepted"], got["path"]]
            assert not ws[:131072].any()
