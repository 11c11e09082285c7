"""Rows with more children than a wave has lanes (include/moe_sample.h), of which one behind the first 64
is accepted, and the distribution of tokens over 16000 sequences; against the float64 oracle and by the
margins of test_gpu_sample.py."""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev, log
from test_gpu_sample import MARGIN, Case, check
from tree_support import tree_of

pytestmark = pytest.mark.gpu


def one_parent(kids, rng, dtype="f32", drawn=False, seqs=1):
    """Sequences of a root with `kids` children."""
    c = Case([kids + 1] * seqs, 3000, kids, rng, dtype, drawn, spread=1.0)
    c.parents = np.tile(np.array([-1] + [0] * kids, np.int32), seqs)
    c.temperature[:] = 1.0
    return c


@pytest.mark.parametrize("kids,taken", [
    (65, [64]), (130, [64]), (130, [100]), (130, [129]), (300, [128]), (300, [299]), (130, [3, 100]), (130, [63, 64]),
    (200, [70, 150, 199]), (130, []),
])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_given_child_behind_the_first_64(kids, taken, dtype):
    """Children with the number 0 are accepted (0 < p), the others all but never: the first of them it is."""
    log(f"given {kids} children, {taken} {dtype}")
    rng = np.random.default_rng(kids + len(taken))
    c = one_parent(kids, rng, dtype, seqs=2)
    for b in range(2):
        c.tokens[b * (kids + 1):(b + 1) * (kids + 1)] = rng.permutation(3000)[:kids + 1]
    c.accept_u[:] = 1 - 2.0 ** -24
    for k in taken:
        c.accept_u[1 + k] = 0.0  # of the first sequence
    got = check(c)
    assert got["n_accepted"] == [int(bool(taken)), 0]
    assert not taken or got["path"][0][1] == 1 + taken[0]


@pytest.mark.parametrize("kids,taken", [(65, 64), (130, 64), (130, 65), (130, 127), (130, 129), (130, None)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_a_drawn_child_behind_the_first_64(kids, taken, dtype):
    """The draft's probabilities lie on other tokens than the target's: a child with one of the draft's tokens
    is rejected, all but never with one of the target's.  The sums of the rejections add up in c: 130 errors of
    1.7e-13, and c up to 130, so what a decision compares is off by less than 1e-8."""
    log(f"drawn {kids} children, {taken} {dtype}")
    rng = np.random.default_rng(kids)
    c = one_parent(kids, rng, dtype, drawn=True, seqs=2)
    x = rng.standard_normal((2 * (kids + 1), 3000))
    x[:, 1500:] += 12.0
    c.set_logits(x, dtype)
    q = np.exp(rng.standard_normal(x.shape))
    q[:, 1500:] *= 1e-6
    c.q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    c.tokens[:] = rng.integers(0, 1500, len(c.tokens))
    c.accept_u[:] = 0.25 + 0.5 * c.accept_u
    if taken is not None:
        c.tokens[1 + taken] = 1500 + int(np.argmax(c.x[0, 1500:]))
    got = check(c, margin=1e-8)
    assert got["n_accepted"] == [int(taken is not None), 0]
    assert taken is None or got["path"][0][1] == 1 + taken


@pytest.mark.parametrize("drawn", [False, True])
def test_a_tree_without_a_number_of_children(drawn):
    """Any child can be accepted."""
    rng = np.random.default_rng(84)
    c = one_parent(7, rng, drawn=drawn, seqs=40)
    x = rng.standard_normal((320, 3000))
    x[:, :20] += 8.0
    c.set_logits(x, "f32")
    q = np.exp(rng.standard_normal(x.shape))
    q[:, :20] *= 400.0
    c.q = (q / q.sum(1, keepdims=True)).astype(np.float32) if drawn else None
    c.tokens[:] = rng.integers(0, 20, len(c.tokens))
    want = c.want()
    assert want["margin"] > MARGIN and max(max(p) for p in want["path"]) > 3
    args, named = c.device()
    accepted, n, path = c.outputs()
    tree = svr.DraftTree(args[0].q_offsets, args[0].parents, 8)
    svr.moe_verify_sample(tree, *args[1:], accepted, n, path, **named)
    assert [accepted.tolist(), n.tolist(), path.tolist()] == [want["accepted"], want["n_accepted"], want["path"]]


@pytest.mark.parametrize("kids,drawn", [(1, True), (3, True), (3, False)])
def test_the_first_tokens_of_16000_sequences(kids, drawn):
    """One pair of distributions, counted over as many calls as it takes."""
    rng = np.random.default_rng(83)
    V, n, rows = 12, 16000 // (1 + kids), 1 + kids
    x = np.log(rng.dirichlet(np.ones(V))).astype(np.float32)
    e = np.exp(x.astype(np.float64))
    p = e / e.sum()
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    t = tree_of(np.arange(n + 1, dtype=np.int32) * rows, np.tile(np.array([-1] + [0] * kids, np.int32), n), rows, kids)
    i32 = dict(dtype=torch.int32, device="cuda")
    accepted, count = torch.empty((n, rows), **i32), torch.empty(n, **i32)
    f = lambda m: dev(rng.random(m).astype(np.float32))  # noqa: E731
    got, of, taken = np.zeros(V, np.int64), 0, 0
    while of < 16000:
        if drawn:
            tokens = rng.choice(V, n * rows, p=q.astype(np.float64) / q.astype(np.float64).sum())
        else:
            tokens = np.tile(np.concatenate([[0], np.argsort(-q)[:kids]]), n)
        svr.moe_verify_sample(t, dev(np.tile(x, (n * rows, 1))), dev(tokens.astype(np.int32)), f(n * rows), f(n), accepted,
                              count, draft_probs=dev(np.tile(q, (n * rows, 1))) if drawn else None)
        got += np.bincount(accepted[:, 0].cpu().numpy(), minlength=V)
        of += n
        taken += int((count > 0).sum())
    # Five standard deviations of each count.
    assert got.sum() == of == 16000 and np.all(np.abs(got - of * p) <= 5 * np.sqrt(of * p * (1 - p)))
    assert 0 < taken < of
