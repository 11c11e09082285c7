"""Log probabilities, entropy and top alternatives (include/moe_logprobs.h) on
the GPU against the float64 oracle, every call through the C ABI."""

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from gpu_common import dev, log
from kv_support import TYPES
from oracle import logprobs_oracle as lo

pytestmark = pytest.mark.gpu


def run(x, targets, k, ws=None):
    """x: device logits [N][V] (rows possibly apart)."""
    N = x.shape[0]
    lp, h = (torch.full((N,), 77.0, device="cuda") for _ in range(2))
    ids = torch.full((N, k), -7, dtype=torch.int32, device="cuda")
    tl = torch.full((N, k), 77.0, device="cuda")
    svr.moe_logprobs(x, dev(np.asarray(targets, np.int32)), lp, h, ids, tl, ws=ws)
    torch.cuda.synchronize()
    return dict(logprobs=lp, entropy=h, top_ids=ids, top_logprobs=tl)


def check(x, targets, k, ws=None):
    """Tolerances: a logit's distance from the maximum is one rounding of 2^-24 of it; z is a sum of V
    positive terms in parts of at most V/64 + 80 terms one after another (a lane's columns, then the
    joins), a term's exponential within 2^-22 + its distance's rounding; its logarithm is off by as
    much absolutely.  The entropy adds sum w |d| / z, whose terms carry the same relative error."""
    got = {n: v.cpu().numpy() for n, v in run(x, targets, k, ws).items()}
    L = x.double().cpu().numpy()
    ref = lo.logprobs(L, targets, k)
    assert np.array_equal(got["top_ids"], ref["top_ids"])
    u = 2.0 ** -24
    V = L.shape[1]
    rel = (V / 64 + 80 + 4 + 200) * u  # 200: d up to 200 in an exponential that matters at all
    for n in ("logprobs", "top_logprobs"):
        r, g = ref[n], got[n].astype(np.float64)
        assert np.array_equal(np.isnan(r), np.isnan(g)) and np.array_equal(np.isinf(r), np.isinf(g)), n
        f = np.isfinite(r)
        assert np.all(np.abs(g[f] - r[f]) <= rel + 4 * u * np.abs(r[f])), n
    r, g = ref["entropy"], got["entropy"].astype(np.float64)
    assert np.array_equal(np.isnan(r), np.isnan(g))
    f = np.isfinite(r)
    assert np.all(np.abs(g[f] - r[f]) <= 2 * rel * (1 + np.abs(r[f])) + 8 * u * 20)
    return got


def draw(rng, N, V, dtype, spread=2.5):
    x = rng.standard_normal((N, V)).astype(np.float32) * spread
    return dev(x).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,k", [
    (1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 63, 5), (5, 1000, 64), (1, 1024, 20), (4, 1025, 20),
    (7, 5001, 8), (4, 131072, 20), (1, 131072, 64), (65, 4097, 3), (600, 2048, 5), (513, 4099, 1),
])
def test_seeded_rows(dtype, N, V, k):
    log(f"logprobs {dtype} N={N} V={V} k={k}")
    rng = np.random.default_rng(N + V)
    check(draw(rng, N, V, dtype), rng.integers(0, V, N), k)


def test_ties_go_to_the_lower_column():
    V = 9000
    x = np.zeros((6, V), np.float32)
    x[1, ::3] = 1.0
    x[2] = np.arange(V) // 50
    x[3] = -(np.arange(V) // 50)
    x[4, [8999, 4096, 4095, 1024, 1023, 5]] = 7.0
    x[5] = -0.0
    x[5, 8000] = 0.0
    for d in ("f32", "bf16", "f16"):
        check(dev(x).to(TYPES[d]), [0, 1, 2, 3, 4, 5], 33)


def test_rising_and_falling_rows():
    """Every column better than all before it, and the reverse: the list is cut again and again."""
    x = np.stack([np.arange(20000), -np.arange(20000), np.arange(20000) % 977]).astype(np.float32) / 16
    check(dev(x), [19999, 0, 5], 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_columns(dtype):
    rng = np.random.default_rng(3)
    V = 5000
    for low in (-np.inf, float(torch.finfo(TYPES[dtype]).min)):
        x = draw(rng, 5, V, dtype)
        x[0, 7:] = low           # seven columns left: alternatives run into the mask
        x[1, :] = low            # none left
        x[2, ::2] = low
        x[3, :4999] = low        # only the last
        x[4, 100] = low
        check(x, [3, 4, 1, 4999, 100], 20)


def test_nan_and_infinity():
    rng = np.random.default_rng(4)
    x = draw(rng, 5, 3000, "f32")
    x[0, 17] = float("nan")
    x[1, :] = float("nan")
    x[2, 5] = float("inf")
    x[3, [9, 2999]] = float("inf")
    got = check(x, [17, 0, 5, 9, 1], 10)
    assert 17 not in got["top_ids"][0] and got["top_ids"][1].tolist() == list(range(10))


def test_targets_outside_the_vocabulary():
    rng = np.random.default_rng(5)
    got = check(draw(rng, 4, 100, "f32"), [-1, 100, 2 ** 31 - 1, 99], 2)
    assert np.isnan(got["logprobs"][:3]).all()


def test_certain_rows():
    x = np.full((3, 1000), -200.0, np.float32)
    x[0, 3] = 0
    x[1, 3], x[1, 4] = 0, -20
    x[2] = 50.0
    check(dev(x), [3, 4, 10], 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_apart_and_unaligned(dtype):
    rng = np.random.default_rng(6)
    for V, width, at in ((5000, 5120, 0), (5000, 5003, 0), (999, 1024, 1), (4096, 4104, 8)):
        buf = draw(rng, 3, width, dtype)
        buf[:] = buf.abs() + 50  # what lies beside the rows would win
        x = buf[:, at:at + V]
        x -= 50
        check(x, [0, 1, 2], 5)


def test_only_some_outputs():
    rng = np.random.default_rng(7)
    x = draw(rng, 3, 2000, "f32")
    full = run(x, [1, 2, 3], 4)
    h = torch.empty(3, device="cuda")
    svr.moe_logprobs(x, None, None, h)
    assert torch.equal(h, full["entropy"])
    ids = torch.empty((3, 4), dtype=torch.int32, device="cuda")
    svr.moe_logprobs(x, None, None, None, ids)
    assert torch.equal(ids, full["top_ids"])
    lp = torch.empty(3, device="cuda")
    svr.moe_logprobs(x, dev(np.array([1, 2, 3], np.int32)), lp)
    assert torch.equal(lp, full["logprobs"])


def test_one_workspace_for_batches_of_every_size():
    rng = np.random.default_rng(8)
    ws = svr.logprobs_workspace(600, 20000, 20)
    for N in (600, 1, 300, 4, 512, 513, 2):
        check(draw(rng, N, 20000 if N < 10 else 5000, "bf16"), rng.integers(0, 5000, N), 20, ws)
        assert int(ws[:2048].count_nonzero().item()) == 0


def test_a_row_beyond_two_gibielements():
    V, stride = 4000, 2 ** 31 + 16
    buf = torch.empty(stride + V, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, V), (stride, 1))
    rng = np.random.default_rng(9)
    x.copy_(draw(rng, 2, V, "bf16"))
    check(x, [5, 6], 5)


def test_replayed_from_a_graph_after_verify_accept():
    """Accept and log probabilities of its tokens in one graph, replayed on changing logits."""
    rng = np.random.default_rng(10)
    M, V, k = 4, 30000, 5
    x = draw(rng, M, V, "f32")
    drafts = dev(np.array([5, 6, 7], np.int32))
    tok, acc, n = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in (M, M, 1))
    lp, h, tl = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros((M, k), device="cuda")
    ids = torch.zeros((M, k), dtype=torch.int32, device="cuda")
    wa, wl = svr.accept_workspace(M, V), svr.logprobs_workspace(M, V, k)

    def step():
        svr.moe_verify_accept(x, drafts, tok, acc, n, ws=wa)
        svr.moe_logprobs(x, tok, lp, h, ids, tl, ws=wl)

    step()
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(4):
        x.copy_(draw(rng, M, V, "f32"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = (tok.clone(), lp.clone(), h.clone(), ids.clone(), tl.clone())
        assert torch.equal(ids[:, 0], tok) and torch.equal(tl[:, 0], lp), i
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (tok, lp, h, ids, tl))), i


def test_workspace_made_on_the_stream_of_the_call():
    rng = np.random.default_rng(61)
    x = draw(rng, 2, 131072, "f32")
    want = run(x, [5, 6], 5)
    side = torch.cuda.Stream()
    got, n = [], svr.moe_logprobs_workspace_bytes(2, 131072, 5)
    t = dev(np.array([5, 6], np.int32))
    for _ in range(20):
        o = {k: torch.empty_like(v) for k, v in want.items()}
        svr.moe_logprobs(x, t, stream=side, **o)
        got.append(o)
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)  # what this stream may be given
    torch.cuda.synchronize()
    for o in got:
        for k, v in want.items():
            assert torch.equal(o[k], v), k


def test_workspace_of_the_call_stays_on_its_stream():
    """Everything but the workspaces is made, and waited for, before the calls: what this stream is given and
    fills meanwhile can only be a workspace's memory, which it must not be."""
    rng = np.random.default_rng(62)
    x = draw(rng, 2, 131072, "f32")
    want = run(x, [5, 6], 5)
    t = dev(np.array([5, 6], np.int32))
    n = svr.moe_logprobs_workspace_bytes(2, 131072, 5)
    got = [{k: torch.zeros_like(v) for k, v in want.items()} for _ in range(20)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for o in got:
        svr.moe_logprobs(x, t, stream=side, **o)
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    for o in got:
        for k, v in want.items():
            assert torch.equal(o[k], v), k
