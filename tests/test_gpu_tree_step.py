"""The operators of a verify step on trees of drafts together, as a serving loop calls them: plan, cache
append, tree attention, the MoE layer, sampled verification and commit, for two sequences at once, eagerly
and replayed from one captured graph.

The model is a toy of one layer with tables for what a user's projections give: a token's embedding and
its fused q/k/v row are looked up, logits are scaled columns of the layer's output.  Everything else is
the library."""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
import synth
from _support import small_config
from gpu_common import desc_of as layer_desc_of, dev, upload
from kv_support import attention_tolerance, desc_of
from oracle import kv_oracle as ko, sample_oracle as so, tree_oracle as to
from tree_support import tree_of

pytestmark = pytest.mark.gpu

V, LAYERS = 777, 2  # caches: the commit moves the path in both
LAY = ko.Layout(8, 2, 64, 16, 0, 64, False)
# Two trees: two children a row, three levels; and a branch beside a chain.
PARENTS = [[-1, 0, 0, 1, 1, 2, 2], [-1, 0, 0, 2]]
PROMPTS = [9, 21]


class Model:
    """Two sequences, their caches, and the static buffers of a step."""

    def __init__(self, parents, pages=12):
        rng = np.random.default_rng(41)
        D, hq, hk = LAY.dim, LAY.heads, LAY.kv_heads
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.rows = [len(p) for p in parents]
        self.parents = np.array([x for p in parents for x in p], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(self.rows)]).astype(np.int32)
        T, B, M = int(self.offsets[-1]), len(parents), max(self.rows)
        self.T, self.B, self.M = T, B, M
        self.cfg = small_config(hidden=512, n_experts=16, top_k=4, ffn=256, shared_ffn=256, expert_type="q4_k",
                                n_tokens=T, seed_index=170)
        H = self.cfg.hidden
        self.emb, self.qkv = f(V, H), f(V, (hq + 2 * hk) * D).bfloat16()
        self.norms = 1 + 0.1 * f(2, D)
        self.columns, self.mult = dev(rng.integers(0, H, V)), f(V)
        self.inv_freq = dev((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
        self.weights = upload(synth.draw_layer(self.cfg))
        self.d, self.ld = desc_of(LAY), layer_desc_of(self.cfg)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = np.array([[5, 2, 7, 0, 11, 9], [3, 1, 6, 4, 10, 8]], np.int32)
        self.lens = torch.zeros(B, **i32)
        self.tree = tree_of(self.offsets, self.parents, M, 2)
        self.batch = svr.KvBatch(dev(self.offsets), self.lens, dev(self.table), M)
        self.caches = [svr.kv_cache(self.d, pages) for _ in range(LAYERS)]
        self.fed = torch.zeros(T, **i32)
        self.mask = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
        self.positions = torch.zeros(T, **i32)
        self.qo = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
        self.att, self.y = torch.empty_like(self.qo), torch.empty((T, H), device="cuda")
        self.logits = torch.empty((T, V), device="cuda")
        self.temperature = torch.zeros(B, device="cuda")
        self.accept_u, self.sample_u = torch.zeros(T, device="cuda"), torch.zeros(B, device="cuda")
        self.probs = torch.zeros((T, V), device="cuda")
        self.acc, self.path = torch.empty((B, M), **i32), torch.empty((B, M), **i32)
        self.n, self.kept = torch.empty(B, **i32), torch.empty(B, **i32)
        self.pending = torch.empty((B, H), device="cuda")
        self.ws = [svr.kv_workspace(self.d, self.batch, T), svr.workspace(self.ld, T),
                   svr.sample_workspace(self.tree, T, V)]

    def launch(self, drawn=False):
        D, hq, hk = LAY.dim, LAY.heads, LAY.kv_heads
        svr.moe_tree_plan(self.tree, self.lens, self.mask, self.positions)
        row = self.qkv[self.fed.long()]
        q, k, v = (t.unflatten(1, (-1, D)) for t in row.split([hq * D, hk * D, hk * D], 1))
        for c in self.caches:
            svr.moe_kv_append(self.d, self.batch, q, k, v, c, self.qo, q_norm=self.norms[0], k_norm=self.norms[1],
                              inv_freq=self.inv_freq, positions=self.positions)
        svr.moe_kv_tree_attention(self.d, self.batch, self.mask, self.qo, self.caches[0], self.att, ws=self.ws[0])
        x = self.emb[self.fed.long()] + self.att.float().flatten(1)
        svr.moe_layer_forward(self.ld, self.weights, x, self.y, None, None, ws=self.ws[1])
        torch.mul(self.y[:, self.columns], self.mult, out=self.logits)
        svr.moe_verify_sample(self.tree, self.logits, self.fed, self.accept_u, self.sample_u, self.acc, self.n,
                              self.path, draft_probs=self.probs if drawn else None, temperature=self.temperature,
                              verify_h=self.y, pending_h=self.pending, ws=self.ws[2])
        svr.moe_kv_commit(self.d, self.batch, self.path, self.n, self.caches, self.kept)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (*self.caches, self.mask, self.positions, self.qo, self.att, self.y, self.logits,
                                    self.acc, self.path, self.n, self.kept, self.pending)]


def check_step(m, before, drawn=False):
    """Each operator's outputs against the oracles, from the inputs that it had."""
    lens = m.lens.cpu().numpy()
    words, pos, _ = to.plan(m.offsets, m.parents, lens, m.M, 1)
    assert np.array_equal(m.mask.cpu().numpy().view(np.uint64), words)
    assert np.array_equal(m.positions.cpu().numpy(), pos)
    # The cache as attention saw it: with the tree's rows, before the commit.
    row = m.qkv[m.fed.long()].double().cpu().numpy()
    D, hq, hk = LAY.dim, LAY.heads, LAY.kv_heads
    q, k, v = (row[:, a:b].reshape(m.T, -1, D) for a, b in ((0, hq * D), (hq * D, (hq + hk) * D),
                                                            ((hq + hk) * D, (hq + 2 * hk) * D)))
    cache = before.cpu().numpy()
    norms = m.norms.cpu().numpy()
    ko.append(LAY, cache, m.offsets, lens, m.table, q, k, v, norms[0], norms[1], m.inv_freq.cpu().numpy(), pos)
    ref, _, size, reach, seen = to.attention(LAY, cache, m.offsets, lens, m.table, m.qo.double().cpu().numpy(), words, m.M)
    tol = attention_tolerance("bf16", ref, size, reach, seen, D)
    assert np.all(np.abs(m.att.double().cpu().numpy() - ref) <= tol)
    host = lambda t: t.cpu().numpy()  # noqa: E731
    want = so.verify(m.logits.double().cpu().numpy(), m.offsets, m.parents, host(m.fed), host(m.accept_u),
                     host(m.sample_u), m.M, 2, host(m.probs) if drawn else None, host(m.temperature))
    assert want["margin"] > 1e-12
    assert m.acc.tolist() == want["accepted"] and m.path.tolist() == want["path"]
    assert m.n.tolist() == want["n_accepted"]
    assert torch.equal(m.pending, m.y[want["row"]])
    kept = to.commit(LAY, cache, m.offsets, lens, m.table, m.M, np.array(want["path"]), want["n_accepted"])
    assert m.kept.tolist() == kept.tolist()
    for c in m.caches:
        assert np.array_equal(host(c), cache)
    return want


def prompts():
    rng = np.random.default_rng(42)
    return [rng.integers(0, V, n).tolist() for n in PROMPTS]


def single_steps(m, fed, lens):
    m.fed.copy_(torch.tensor(fed, dtype=torch.int32))
    m.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    m.launch()
    torch.cuda.synchronize()
    return [a[0] for a in m.acc.tolist()]


def greedy(count):
    """`count` tokens of each sequence made one at a time, and the model that made them."""
    m = Model([[-1], [-1]])
    text = prompts()
    # The shorter prompt ends first: its sequence repeats its last place meanwhile.
    last = None
    for i in range(max(PROMPTS)):
        at = [min(i, n - 1) for n in PROMPTS]
        last = single_steps(m, [s[a] for s, a in zip(text, at)], [a + 1 for a in at])
    made = [[t] for t in last]
    for i in range(count):
        nxt = single_steps(m, [s[-1] for s in made], [n + i + 1 for n in PROMPTS])
        for s, t in zip(made, nxt):
            s.append(t)
    return m, made


def drafts(want, parents, right, rng):
    """A tree's tokens: the next ones of `want` along a branch for `right` levels, others elsewhere."""
    tokens = [want[0]] + [None] * (len(parents) - 1)
    on = 0
    for level in range(right):
        kids = [j for j in range(1, len(parents)) if parents[j] == on]
        if not kids:
            break
        on = kids[int(rng.integers(len(kids)))]
        tokens[on] = want[level + 1]
    for j in range(1, len(parents)):
        if tokens[j] is None:
            tokens[j] = int(rng.integers(V))
    return tokens


def test_tree_steps_make_the_tokens_of_single_ones():
    """Greedy: whatever is drafted, the tokens are those made one at a time, and the committed caches hold
    the same bytes."""
    count = 20
    single, want = greedy(count + 4)
    m = Model(PARENTS)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    m.launch()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        m.launch()
    # The prompts' caches: theirs and nothing else.
    start_cache = single.caches[0].clone()
    for c in m.caches:
        c.copy_(start_cache)
    made, rng, lengths = [[w[0]] for w in want], np.random.default_rng(43), set()
    step = 0
    while min(len(s) for s in made) <= count:
        places = [n + len(s) - 1 for n, s in zip(PROMPTS, made)]
        fed = []
        for b in range(2):
            at = len(made[b]) - 1
            ahead = (want[b][at:] + [0] * 4)[:4]
            fed += drafts(ahead, PARENTS[b], (step + b) % 4, rng)
        m.fed.copy_(torch.tensor(fed, dtype=torch.int32))
        m.lens.copy_(torch.tensor([p + r for p, r in zip(places, m.rows)], dtype=torch.int32))
        before = [c.clone() for c in m.caches]
        m.launch()
        eager = m.outputs()
        check_step(m, before[0])
        for c, b in zip(m.caches, before):
            c.copy_(b)
        for t in (m.att, m.y, m.logits):
            t.fill_(float("nan"))
        g.replay()
        for a, b in zip(eager, m.outputs()):
            assert torch.equal(a, b)
        for b in range(2):
            n = int(m.n[b])
            lengths.add(n)
            made[b] += m.acc[b, :n + 1].tolist()
        step += 1
    assert all(s[:count] == w[:count] for s, w in zip(made, want))
    assert lengths == {0, 1, 2}
    # Read back, the committed places hold what the single steps stored.
    n = [p + count - 1 for p in PROMPTS]
    batch = svr.KvBatch(dev(np.array([0, n[0], sum(n)], np.int32)), dev(np.array(n, np.int32)), dev(m.table), max(n))
    out = [[torch.empty((sum(n), LAY.kv_heads, LAY.dim), device="cuda") for _ in "kv"] for _ in range(2)]
    svr.moe_kv_read(m.d, batch, m.caches[1], *out[0])
    svr.moe_kv_read(m.d, batch, single.caches[0], *out[1])
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("drawn", [False, True])
def test_sampled_tree_steps(drawn):
    """With temperatures, drafts given or drawn: every step against the oracles, eagerly and replayed."""
    m = Model(PARENTS)
    rng = np.random.default_rng(44)
    for c in m.caches:
        c.copy_(greedy(0)[0].caches[0])
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    m.lens.copy_(torch.tensor([n + r for n, r in zip(PROMPTS, m.rows)], dtype=torch.int32))
    before = [c.clone() for c in m.caches]
    m.launch(drawn)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        m.launch(drawn)
    for c, b in zip(m.caches, before):
        c.copy_(b)
    lens, roots, counts = list(PROMPTS), [3, 5], []
    m.temperature.copy_(torch.tensor([0.8, 1.3]))
    for step in range(10):
        # Drafts from some distribution: flat over a few tokens; the first step's rows show likely ones.
        q = np.zeros((m.T, V), np.float32)
        likely = m.logits.cpu().numpy().argsort(1)[:, -6:]
        for i in range(m.T):
            q[i, likely[i]] = 1 / 6
        fed = []
        for b in range(2):
            off = int(m.offsets[b])
            for j in range(m.rows[b]):
                fed.append(roots[b] if j == 0 else int(rng.choice(V, p=q[off + PARENTS[b][j]] / q[off + PARENTS[b][j]].sum())))
        m.probs.copy_(dev(q))
        m.fed.copy_(torch.tensor(fed, dtype=torch.int32))
        m.accept_u.copy_(dev(rng.random(m.T).astype(np.float32)))
        m.sample_u.copy_(dev(rng.random(2).astype(np.float32)))
        m.lens.copy_(torch.tensor([n + r for n, r in zip(lens, m.rows)], dtype=torch.int32))
        before = [c.clone() for c in m.caches]
        m.launch(drawn)
        eager = m.outputs()
        want = check_step(m, before[0], drawn)
        for c, b in zip(m.caches, before):
            c.copy_(b)
        g.replay()
        for a, b in zip(eager, m.outputs()):
            assert torch.equal(a, b)
        counts += want["n_accepted"]
        lens = m.kept.tolist()
        roots = [want["accepted"][b][want["n_accepted"][b]] for b in range(2)]
    assert lens == [p + 10 + sum(counts[b::2]) for b, p in enumerate(PROMPTS)]
