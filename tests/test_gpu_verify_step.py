"""The operators of a verify step together, as a serving loop calls them: cache append, attention, the
MoE layer, verify/accept and log probabilities, eagerly and replayed from one captured graph.

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
from oracle import accept_oracle as ao, kv_oracle as ko, logprobs_oracle as lo
from kv_support import attention_tolerance, desc_of

pytestmark = pytest.mark.gpu

V, PROMPT, DRAFTS = 777, 9, 3
LAY = ko.Layout(8, 2, 64, 16, 0, 64, False)
CFG = small_config(hidden=512, n_experts=16, top_k=4, ffn=256, shared_ffn=256, expert_type="q4_k",
                   n_tokens=DRAFTS + 1, seed_index=170)


class Model:
    """One sequence, its cache, and the static buffers of a step of M rows."""

    def __init__(self, M, pages=8):
        rng = np.random.default_rng(41)
        D, hq, hk = LAY.dim, LAY.heads, LAY.kv_heads
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.M = M
        self.emb, self.qkv = f(V, CFG.hidden), f(V, (hq + 2 * hk) * D).bfloat16()
        self.norms = 1 + 0.1 * f(2, D)
        self.columns, self.mult = dev(rng.integers(0, CFG.hidden, V)), f(V)
        self.inv_freq = dev((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
        self.weights = upload(synth.draw_layer(CFG))
        self.d, self.ld = desc_of(LAY), layer_desc_of(CFG)
        i32 = dict(dtype=torch.int32, device="cuda")
        table = torch.tensor([[5, 2, 7, 0, 3, 1, 6, 4][:pages]], **i32)
        self.lens = torch.zeros(1, **i32)
        self.batch = svr.KvBatch(torch.tensor([0, M], **i32), self.lens, table, M)
        self.table = table.cpu().numpy()
        self.cache = svr.kv_cache(self.d, pages)
        self.fed = torch.zeros(M, **i32)
        self.qo = torch.empty((M, hq, D), dtype=torch.bfloat16, device="cuda")
        self.att = torch.empty_like(self.qo)
        self.y = torch.empty((M, CFG.hidden), device="cuda")
        self.logits = torch.empty((M, V), device="cuda")
        self.tok, self.acc, self.n = torch.empty(M, **i32), torch.empty(M, **i32), torch.empty(1, **i32)
        self.lp, self.ent = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        self.ids, self.top = torch.empty((M, 5), **i32), torch.empty((M, 5), device="cuda")
        self.ws = [svr.kv_workspace(self.d, self.batch, M), svr.workspace(self.ld, M),
                   svr.accept_workspace(M, V), svr.logprobs_workspace(M, V, 5)]

    def launch(self):
        D, hq, hk = LAY.dim, LAY.heads, LAY.kv_heads
        row = self.qkv[self.fed.long()]
        q, k, v = (t.unflatten(1, (-1, D)) for t in row.split([hq * D, hk * D, hk * D], 1))
        svr.moe_kv_append(self.d, self.batch, q, k, v, self.cache, self.qo, q_norm=self.norms[0],
                          k_norm=self.norms[1], inv_freq=self.inv_freq)
        svr.moe_kv_attention(self.d, self.batch, self.qo, self.cache, self.att, ws=self.ws[0])
        x = self.emb[self.fed.long()] + self.att.float().flatten(1)
        svr.moe_layer_forward(self.ld, self.weights, x, self.y, None, None, ws=self.ws[1])
        torch.mul(self.y[:, self.columns], self.mult, out=self.logits)
        svr.moe_verify_accept(self.logits, self.fed[1:] if self.M > 1 else None, self.tok, self.acc, self.n,
                              ws=self.ws[2])
        svr.moe_logprobs(self.logits, self.tok, self.lp, self.ent, self.ids, self.top, ws=self.ws[3])

    def feed(self, tokens, place):
        """The tokens at places [place, place + M)."""
        self.fed.copy_(torch.tensor(tokens, dtype=torch.int32))
        self.lens.fill_(place + self.M)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.cache, self.qo, self.att, self.y, self.logits, self.tok, self.n,
                                    self.lp, self.ent, self.ids, self.top)]


def start():
    """The prompt, and its cache and first token."""
    prompt = np.random.default_rng(42).integers(0, V, PROMPT).tolist()
    m = Model(PROMPT)
    m.feed(prompt, 0)
    m.launch()
    torch.cuda.synchronize()
    return prompt, m.cache, int(m.tok[-1])


def greedy(count):
    """Tokens made one at a time."""
    prompt, cache, token = start()
    m = Model(1)
    m.cache.copy_(cache)
    out = [token]
    for i in range(count):
        m.feed(out[-1:], PROMPT + i)
        m.launch()
        torch.cuda.synchronize()
        out.append(int(m.tok[0]))
    return out


def check_step(m, place):
    """Each operator's outputs against the oracles, from the inputs that it had."""
    cache = m.cache.cpu().numpy()
    q = m.qo.double().cpu().numpy()
    ref, _, size, reach, seen = ko.attention(LAY, cache, [0, m.M], [place + m.M], m.table, q)
    tol = attention_tolerance("bf16", ref, size, reach, seen, LAY.dim)
    assert np.all(np.abs(m.att.double().cpu().numpy() - ref) <= tol)
    L = m.logits.cpu().numpy()
    want = ao.verify_accept(L, m.fed[1:].cpu().numpy())
    assert m.tok.tolist() == want["tokens"] and int(m.n) == want["n_accepted"]
    lp = lo.logprobs(L.astype(np.float64), want["tokens"], 5)
    assert np.array_equal(m.ids.cpu().numpy(), lp["top_ids"])
    # The token is the best alternative: the same number, twice.
    assert torch.equal(m.lp, m.top[:, 0]) and torch.equal(m.tok, m.ids[:, 0])
    u = 2.0 ** -24  # as in the operator's own tests
    assert np.all(np.abs(m.lp.cpu().numpy() - lp["logprobs"]) <= (V / 64 + 284) * u + 4 * u * np.abs(lp["logprobs"]))


def test_verify_steps_make_the_tokens_of_single_ones():
    """Drafts right, wrong from some place on, or all wrong: the accepted tokens are the greedy ones, and
    rejected rows of the cache are overwritten by the next step."""
    count = 24
    want = greedy(count + DRAFTS + 1)
    prompt, cache, token = start()
    assert token == want[0]
    m = Model(DRAFTS + 1)
    m.cache.copy_(cache)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    m.feed([0] * m.M, 0)
    m.launch()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        m.launch()
    m.cache.copy_(cache)
    made, step, counts = [token], 0, []
    while len(made) <= count:
        right = step % (DRAFTS + 2)
        at = len(made)
        drafts = [t if j < right else (t + 1) % V for j, t in enumerate(want[at:at + DRAFTS])]
        place = PROMPT + at - 1
        before = m.cache.clone()
        m.feed([made[-1]] + drafts, place)
        m.launch()
        eager = m.outputs()
        check_step(m, place)
        m.cache.copy_(before)
        for t in (m.att, m.y, m.logits, m.lp):
            t.fill_(float("nan"))
        g.replay()
        for a, b in zip(eager, m.outputs()):
            assert torch.equal(a, b)
        n = int(m.n)
        counts.append(n)
        made += m.tok[:n + 1].tolist()
        step += 1
    assert made[:count] == want[:count]
    assert set(counts) == set(range(DRAFTS + 1))
