"""Cases of a verify step on a tree of drafted tokens, and the operators' plain forms.

Four operators, in the order of a step: the tree's plan (which rows see which, and
at what positions), attention of the tree's rows over the paged 4-bit cache,
verification of the drafts against the target's probabilities from given random
numbers, and the move of the accepted path's tokens to their places in the cache.
Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU,
``run`` makes one pass: with ``own`` the framework's calls, without it elementary
torch operations in 32 bits (64 for the verification, whose cumulative sums have a
border every millionth).
"""

from __future__ import annotations

import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# Values of the 4-bit codes (E2M1): bit 3 is the sign.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# The most a drawn case may cost: what the largest listed ones cost.
MOST_PAIRS = 61 * 64 * 60000 * 192  # query rows x heads x visible tokens x head size
MOST_CACHE = 60000 * 4 * 192        # tokens x KV heads x head size
MOST_LOGITS = 200 * 131072
MOST_PLAN = 48 * 253
MOST_MOVED = 48 * 8 * 6 * 8 * 128   # sequences x KV heads x tokens x layers x head size


def listed():
    p, t = dict(op="plan"), dict(op="attention", window=0, ragged=False)
    v = dict(op="sample", masked=False, greedy=0.0, hidden=0)
    c = dict(op="commit")
    return [
        # One drafted tree of a single request.
        dict(p, name="plan_m61", seqs=1, rows=61, kids=8, ragged=False),
        # Many requests, trees of uneven size.
        dict(p, name="plan_b48", seqs=48, rows=253, kids=10, ragged=True),
        # A small tree on a short cache: latency counts.
        dict(t, name="tree_m7_short", dtype="bf16", heads=64, kv_heads=4, dim=192, page=64,
             seqs=1, rows=7, kids=3, length=777),
        # A tree of 61 rows on a prompt of 60000 tokens.
        dict(t, name="tree_m61_60000", dtype="bf16", heads=64, kv_heads=4, dim=192, page=64,
             seqs=1, rows=61, kids=8, length=60000),
        # Many requests of uneven lengths and trees, small pages.
        dict(t, name="tree_b29_ragged", dtype="f16", heads=32, kv_heads=8, dim=128, page=16,
             seqs=29, rows=26, kids=4, length=5000, ragged=True),
        # A sliding-window layer in 32-bit activations.
        dict(t, name="tree_window_512", dtype="f32", heads=64, kv_heads=4, dim=192, page=64,
             seqs=8, rows=13, kids=4, length=6001, ragged=True, window=512),
        # The verify batch of a chain of three given drafts, with the hidden state kept.
        dict(v, name="sample_m4", dtype="f32", vocab=131072, seqs=1, rows=4, kids=1, drawn=False,
             ragged=False, hidden=4096),
        # Many requests, chains drawn from the drafts' own probabilities, some requests greedy.
        dict(v, name="sample_chain_b48", dtype="bf16", vocab=131072, seqs=48, rows=5, kids=1,
             drawn=True, ragged=True, greedy=0.2),
        # A tree of given drafts (the draft model's best tokens), under a grammar's mask.
        dict(v, name="sample_tree_m61", dtype="f32", vocab=131072, seqs=1, rows=61, kids=8,
             drawn=False, ragged=False, masked=True),
        # Trees whose siblings are drawn from one distribution, several requests.
        dict(v, name="sample_tree_b9", dtype="f16", vocab=128000, seqs=9, rows=21, kids=3,
             drawn=True, ragged=True),
        # The accepted path of one request in one layer's cache.
        dict(c, name="commit_m61", heads=64, kv_heads=4, dim=192, page=64, seqs=1, rows=61, keep=5,
             length=60000, layers=1),
        # Many requests, the caches of eight layers.
        dict(c, name="commit_b48", heads=32, kv_heads=8, dim=128, page=16, seqs=48, rows=26, keep=5,
             length=3000, layers=8),
    ]


def _log_int(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["plan", "attention", "attention", "sample", "sample", "commit"])
    if op == "plan":
        rows = _log_int(rng, 1, 1000)
        return dict(op=op, seqs=_log_int(rng, 1, max(1, MOST_PLAN // rows)), rows=rows,
                    kids=rng.choice([1, 2, 4, 10]), ragged=rng.random() < 0.6)
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "sample":
        vocab, drawn = _log_int(rng, 1000, 262144), rng.random() < 0.5
        kids = rng.choice([1, 1, 2, 3]) if drawn else rng.choice([1, 1, 2, 4, 10])
        rows = _log_int(rng, 1, 8 if kids == 1 else 64)
        rows = max(1, min(rows, MOST_LOGITS // (2 * vocab)))
        return dict(op=op, dtype=dtype, vocab=vocab,
                    seqs=_log_int(rng, 1, max(1, min(256, MOST_LOGITS // (2 * rows * vocab)))),
                    rows=rows, kids=kids, drawn=drawn, ragged=rng.random() < 0.6,
                    masked=rng.random() < 0.3, greedy=rng.choice([0.0, 0.0, 0.3]),
                    hidden=rng.choice([0, 0, 4096]))
    dim = rng.choice([64, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    rows = _log_int(rng, 1, 100)
    if op == "commit":
        keep, layers = rng.choice([0, 1, 3, 5]), rng.choice([1, 2, 4, 8])
        most = MOST_MOVED // (2 * kv_heads * dim * layers * (keep + 1))
        return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, rows=rows, keep=keep,
                    seqs=_log_int(rng, 1, max(1, min(48, most))),
                    length=rows + _log_int(rng, 1, 3000), layers=layers)
    seqs = _log_int(rng, 1, 32)
    length = rows + _log_int(rng, 1, max(64, min(60000, MOST_CACHE // (seqs * kv_heads * dim))))
    if dtype == "f32":
        length = min(length, rows + 20000)
    rows = max(1, min(rows, MOST_PAIRS // (4 * seqs * heads * length * dim)))
    return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                window=rng.choice([0, 0, 0, 512, 100]), seqs=seqs, rows=rows,
                kids=rng.choice([1, 2, 4, 10]), length=length, ragged=rng.random() < 0.6)


def _tree(rows, kids, rng):
    """Parents of a tree of that many rows, level by level, at most `kids` children a row; row 0 is
    the root (-1).  kids == 1: a chain."""
    parent, free = [-1], [kids]
    open_ = [0]
    for j in range(1, rows):
        # The larger of two: trees that grow deeper than they would by chance.
        p = open_[max(rng.randrange(len(open_)), rng.randrange(len(open_)))]
        parent.append(p)
        free.append(kids)
        open_.append(j)
        free[p] -= 1
        if not free[p]:
            open_.remove(p)
    depth = [0] * rows
    for j in range(1, rows):
        depth[j] = depth[parent[j]] + 1
    order = sorted(range(rows), key=lambda j: (depth[j], j))
    new = {j: i for i, j in enumerate(order)}
    return [-1] + [new[parent[j]] for j in order[1:]]


def _plan(case):
    """Rows, parents and lengths (with the new rows) of every sequence: the case's own, whatever the seed."""
    n, rows, kids, length = case["seqs"], case["rows"], case.get("kids", 1), case.get("length", 0)
    rng = random.Random(n * 1000003 + rows * 8191 + length * 17 + kids)
    ragged = case.get("ragged", False)
    r = [rows] + [rng.randint(1, rows) if ragged else rows for _ in range(n - 1)]
    lens = [length] + [rng.randint(max(x, length // 16, 1), max(x, length)) if ragged else length
                       for x in r[1:]]
    return r, [_tree(x, kids, rng) for x in r], lens


def _ancestors(parents):
    """For every row the rows it sees: its ancestors and itself."""
    seen = []
    for j, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else []) + [j])
    return seen


def _masks(trees, words):
    """The rows' masks as 64-bit words, bit j of row i set where row i sees row j."""
    out = []
    for parents in trees:
        for seen in _ancestors(parents):
            bits = sum(1 << j for j in seen)
            row = [bits >> 64 * w & (1 << 64) - 1 for w in range(words)]
            out.append([x - (1 << 64) if x >> 63 else x for x in row])
    return torch.tensor(out, dtype=torch.int64).view(-1, words)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _page_bytes(dim, page):
    """Codes of keys, codes of values (4 bits each), scales of keys, scales of values (a byte for 32)."""
    return page * (dim + dim // 16)


def _offsets(rows):
    at = [0]
    for r in rows:
        at.append(at[-1] + r)
    return at


def _kept(case):
    """Accepted paths of a commit case: rows in ascending order behind the path's own places, as those
    of a tree with wide first levels are."""
    rng = random.Random(case["seqs"] * 31 + case["rows"])
    paths = []
    for _ in range(case["seqs"]):
        n = min(rng.randint(0, case["keep"]) if case["seqs"] > 1 else case["keep"], (case["rows"] - 1) // 2)
        paths.append([0] + sorted(rng.sample(range(n + 1, case["rows"]), n)))
    return paths


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)

    rows, trees, lens = _plan(case)
    s = dict(case=case, offsets=_int32(_offsets(rows)), max_rows=max(rows), kids=case.get("kids", 1),
             parents=_int32([p for t in trees for p in t]))
    T, B, M = sum(rows), len(rows), max(rows)
    if case["op"] == "plan":
        # The requests' lengths, with the trees' rows.
        more = torch.randint(0, 60000, (B,), generator=g, device="cuda")
        s["lens"] = (more + torch.tensor(rows, device="cuda")).int()
        s["mask"] = torch.empty((T, -(-M // 64)), dtype=torch.int64, device="cuda")
        s["positions"] = torch.empty(T, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "sample":
        return _prepare_sample(s, g, normal, uniform, rows, trees)

    Hq, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    width = -(-max(lens) // P)
    used = [-(-x // P) for x in lens]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    first = _offsets(used)
    take = torch.tensor([[first[b] + min(i, used[b] - 1) for i in range(width)] for b in range(B)],
                        device="cuda")
    s |= dict(lens=_int32(lens), table=order[take])

    def cache():
        codes, scales = _quantise(normal(n_pages, 2, Hk, P, D))
        packed = (codes[..., 0::2] | codes[..., 1::2] << 4).transpose(1, 2).reshape(n_pages, Hk, -1)
        return torch.cat([packed, scales.transpose(1, 2).reshape(n_pages, Hk, -1)], 2).contiguous()

    if case["op"] == "attention":
        s["mask"] = _masks(trees, -(-M // 64)).cuda()
        s["q"] = normal(T, Hq, D).to(TYPES[case["dtype"]])
        s["cache"] = cache()
        s["out"] = torch.empty_like(s["q"])
        return s
    paths = _kept(case)
    wide = max(len(p) for p in paths)
    s["path"] = _int32([p + [-1] * (wide - len(p)) for p in paths])
    s["n_accepted"] = _int32([len(p) - 1 for p in paths])
    s["caches"] = [cache() for _ in range(case["layers"])]
    s["kept"] = torch.empty(B, dtype=torch.int32, device="cuda")
    # To read the committed rows back.
    s["kept_offsets"] = _int32(_offsets([len(p) for p in paths]))
    s["kept_lens"] = _int32([n - r + len(p) for n, r, p in zip(lens, rows, paths)])
    s["max_kept"] = wide
    shape = (sum(len(p) for p in paths), Hk, D)
    s["k_out"], s["v_out"] = ([torch.empty(shape, device="cuda") for _ in s["caches"]] for _ in range(2))
    return s


def _prepare_sample(s, g, normal, uniform, rows, trees):
    case = s["case"]
    V, T, B, M = case["vocab"], sum(rows), len(rows), max(rows)
    x = normal(T, V).mul_(2.5)
    # A few likely tokens on top of the bulk, as a trained model gives.
    likely = torch.randint(0, V, (T, 8), generator=g, device="cuda")
    x.scatter_add_(1, likely, 8.0 + 3.0 * normal(T, 8))
    if case["masked"]:
        keep = uniform(T, V) < 0.1
        keep.scatter_(1, x.argmax(1, keepdim=True), True)
        x.masked_fill_(~keep, float("-inf"))
        del keep
    # Requests differ in temperature; some take the most likely token.
    temperature = 0.7 + 0.6 * uniform(B)
    if case["greedy"]:
        temperature = torch.where(uniform(B) < case["greedy"], torch.zeros_like(temperature), temperature)
    # The draft model's view of the same rows: close to the target's.
    y = x + 0.5 * normal(T, V)
    first = _offsets(rows)
    up = torch.tensor([first[b] + max(p, 0) for b, t in enumerate(trees) for p in t], device="cuda")
    nth, taken = [], {}
    for b, t in enumerate(trees):
        for p in t:
            taken[b, p] = taken.get((b, p), -1) + 1
            nth.append(taken[b, p])
    nth = torch.tensor(nth, device="cuda")
    if case["drawn"]:
        q = torch.softmax(y, -1)
        best = torch.multinomial(q, case["kids"], replacement=True, generator=g)
        s["draft_probs"] = q
    else:
        s["draft_probs"] = None
        best = y.topk(case["kids"], -1).indices
    s["tokens"] = best[up, nth.clamp(max=case["kids"] - 1)].int()
    s["logits"] = x.to(TYPES[case["dtype"]])
    s["temperature"] = temperature
    s["accept_u"], s["sample_u"] = uniform(T), uniform(B)
    s["depth"] = max(len(a) for t in trees for a in _ancestors(t))
    s["accepted"], s["path"] = (torch.empty((B, M), dtype=torch.int32, device="cuda") for _ in range(2))
    s["n_accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["verify_h"] = s["pending_h"] = None
    if case["hidden"]:
        s["verify_h"] = normal(T, case["hidden"])
        s["pending_h"] = torch.empty((B, case["hidden"]), device="cuda")
    if case["kids"] == 1:
        s["parents"] = None  # a chain needs none
    return s


def _quantise(x):
    """4-bit codes and scale bytes of blocks of 32 along the last axis: the scale is the least power
    of two with max|x| <= 7 of it, the code the nearest of E2M1, the even one between two."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 3, e - 2).clamp(-126, 125)
    t = torch.ldexp(b, -e[..., None])
    a = t.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = code | (t < 0).byte() << 3
    return code.flatten(-2), (e + 127).byte()


def _values(codes, scales):
    """The values that codes and scale bytes stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[codes.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(v, scales[..., None].int() - 127).flatten(-2)


def _parts(cache, D, P):
    """Views of a cache: codes of keys and of values, scales of keys and of values."""
    c, s = P * D // 2, P * D // 32
    k, v, ks, vs = cache.split([c, c, s, s], 2)
    return (k.unflatten(2, (P, D // 2)), v.unflatten(2, (P, D // 2)),
            ks.unflatten(2, (P, D // 32)), vs.unflatten(2, (P, D // 32)))


def _sequence(offsets, T):
    """The sequence of every row, and the row's place among its rows."""
    i = torch.arange(T, device=offsets.device)
    b = torch.searchsorted(offsets.long(), i, right=True) - 1
    return b, i - offsets[b]


def _tree_plan(s):
    T, words = s["mask"].shape
    b, at = _sequence(s["offsets"], T)
    up = torch.where(at > 0, s["offsets"][b] + s["parents"], -1).long()
    seen = torch.zeros((T, 64 * words), dtype=torch.bool, device="cuda")
    node, i = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    depth = torch.zeros(T, dtype=torch.int32, device="cuda")
    # A level at a time towards the roots, all rows at once.
    for _ in range(s["max_rows"]):
        on = node >= 0
        where = node.clamp(min=0)
        seen[i, at[where]] |= on
        up_on = on & (up[where] >= 0)
        depth += up_on.int()
        node = torch.where(up_on, up[where], -1)
    bits = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(64, device="cuda")
    mask = (seen.view(T, words, 64).long() * bits).sum(-1)
    base = s["lens"] - (s["offsets"][1:] - s["offsets"][:-1])
    return dict(mask=mask, positions=base[b] + depth)


def _attention(s):
    case = s["case"]
    D, P, W, Hk = case["dim"], case["page"], case["window"], case["kv_heads"]
    T, Hq, _ = s["q"].shape
    B, R = s["lens"].shape[0], s["max_rows"]
    j = torch.arange(R, device="cuda")
    rows = s["offsets"][1:] - s["offsets"][:-1]
    i = (s["offsets"][:-1, None] + j).clamp(max=T - 1).long()
    q = s["q"][i].float().view(B, R, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    kc, vc, ks, vs = (p[s["table"].long()].transpose(2, 3).flatten(1, 2)
                      for p in _parts(s["cache"], D, P))  # [B][tokens][KV heads][...]

    def wide(c, e):
        return _values(torch.stack([c & 15, c >> 4], -1).flatten(-2), e).permute(0, 2, 1, 3)

    n = kc.shape[1]
    base = s["lens"] - rows
    t = torch.arange(n, device="cuda")
    # Marked new rows as columns of the rows' tokens.
    marks = (s["mask"][i][..., None] >> torch.arange(64, device="cuda") & 1).flatten(-2)[..., :R].bool()
    marks &= j < rows[:, None, None]
    new = t - base[:, None]  # token t as a new row
    see = (new < 0)[:, None] | marks.gather(2, new.clamp(0, R - 1)[:, None].expand(B, R, n)) & (
        (new >= 0) & (new < R))[:, None]
    if W:  # the last W tokens that the row sees
        behind = see.flip(-1).cumsum(-1).flip(-1)
        see &= behind <= W
    see = see[:, None, :, None].expand(B, 1, R, Hq // Hk, n).reshape(B, 1, R * (Hq // Hk), n)
    x = (q @ wide(kc, ks).transpose(2, 3)).mul_(D ** -0.5).masked_fill_(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = x.sub_(m.masked_fill(m == float("-inf"), 0.0)).exp_()
    o = (e @ wide(vc, vs)) / e.sum(-1, keepdim=True).clamp_min(1e-37)
    o = o.view(B, Hk, R, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D)
    return o[j < rows[:, None]].to(s["q"].dtype)


def _children(s, T):
    """Row numbers [T][kids] of every row's children, -1 where there are fewer."""
    b, at = _sequence(s["offsets"], T)
    up = at - 1 if s["parents"] is None else s["parents"].long()
    up = torch.where(at > 0, s["offsets"][b] + up, T)
    order = torch.sort(up, stable=True).indices
    own_up = up[order]
    nth = torch.arange(T, device="cuda") - torch.searchsorted(own_up, own_up)
    table = torch.full((T + 1, s["kids"]), -1, device="cuda")
    table[own_up, nth.clamp(max=s["kids"] - 1)] = order
    return b, table[:T]


def _sample(s):
    T = s["logits"].shape[0]
    B, M = s["accepted"].shape
    b, kids = _children(s, T)
    temperature = s["temperature"][b].double()[:, None]
    greedy = temperature[:, 0] <= 0
    x = s["logits"].double()
    d = x - x.amax(-1, keepdim=True)
    e = (d / torch.where(greedy[:, None], 1.0, temperature)).exp_()
    hot = torch.zeros_like(e).scatter_(1, x.argmax(-1, keepdim=True), 1.0)
    p = torch.where(greedy[:, None], hot, e / e.sum(-1, keepdim=True))
    del x, d, e, hot
    w, q = p.clone(), s["draft_probs"]
    left = torch.ones(T, dtype=torch.float64, device="cuda")   # mass of w
    share = torch.zeros(T, dtype=torch.float64, device="cuda")  # of the draft's probabilities taken off
    chosen = torch.full((T,), -1, device="cuda")
    r = torch.arange(T, device="cuda")
    for k in range(kids.shape[1]):
        c = kids[:, k].clamp(min=0)
        col = s["tokens"][c].long()
        here = w[r, col]
        ask = s["accept_u"][c].double() * left
        if q is not None:
            ask = ask * q[r, col].double()
        tried = (kids[:, k] >= 0) & (chosen < 0)
        ok = tried & torch.where(greedy, here > 0, ask < here)
        chosen = torch.where(ok, c, chosen)
        lost = tried & ~ok & ~greedy
        if q is None:
            left = torch.where(lost, left - here, left)
            w[r, col] = torch.where(lost, 0.0, here)
        else:
            share = torch.where(lost, share + left, share)
            less = (p - share[:, None] * q).clamp_min_(0.0)
            w = torch.where(lost[:, None], less, w)
            left = torch.where(lost, less.sum(-1), left)
    at = s["offsets"][:-1].long()
    row = torch.arange(B, device="cuda")
    path, accepted = (torch.full((B, M), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    for _ in range(s["depth"] - 1):
        to = chosen[at]
        go = to >= 0
        nxt = torch.where(go, to, at)
        old = accepted[row, n.long()]
        accepted[row, n.long()] = torch.where(go, s["tokens"][nxt], old)
        n += go.int()
        path[row, n.long()] = (nxt - s["offsets"][:-1]).int()
        at = nxt
    cum = w[at].cumsum(-1)
    token = (cum > s["sample_u"].double()[:, None] * cum[:, -1:]).int().argmax(-1)
    accepted[row, n.long()] = token.int()
    out = dict(accepted=accepted, path=path, n_accepted=n)
    if s["verify_h"] is not None:
        out["pending_h"] = s["verify_h"][at]
    return out


def _commit(s):
    case = s["case"]
    D, P = case["dim"], case["page"]
    base = s["lens"] - (s["offsets"][1:] - s["offsets"][:-1])
    b, i = _sequence(s["kept_offsets"], s["k_out"][0].shape[0])
    b = b.long()
    src, dst = (base[b] + s["path"][b, i.long()]).long(), (base[b] + i).long()
    k_out, v_out = [], []
    for cache in s["caches"]:
        parts = _parts(cache, D, P)
        moved = [part[s["table"][b, src // P].long(), :, src % P] for part in parts]
        for part, new in zip(parts, moved):
            part[s["table"][b, dst // P].long(), :, dst % P] = new
        for out, c, e in ((k_out, moved[0], moved[2]), (v_out, moved[1], moved[3])):
            out.append(_values(torch.stack([c & 15, c >> 4], -1).flatten(-2), e))
    return dict(k=k_out, v=v_out, kept=base + s["n_accepted"] + 1)


def _own(s):
    import speculative_verify_router_amd as svr
    case = s["case"]
    if "tree" not in s:
        s["tree"] = svr.DraftTree(s["offsets"], s["parents"], s["max_rows"], s["kids"])
    if case["op"] == "plan":
        svr.moe_tree_plan(s["tree"], s["lens"], s["mask"], s["positions"])
        return dict(mask=s["mask"], positions=s["positions"])
    if case["op"] == "sample":
        if "ws" not in s:
            s["ws"] = svr.sample_workspace(s["tree"], s["logits"].shape[0], case["vocab"])
        svr.moe_verify_sample(s["tree"], s["logits"], s["tokens"], s["accept_u"], s["sample_u"],
                              s["accepted"], s["n_accepted"], s["path"], draft_probs=s["draft_probs"],
                              temperature=s["temperature"], verify_h=s["verify_h"],
                              pending_h=s["pending_h"], ws=s["ws"])
        out = dict(accepted=s["accepted"], path=s["path"], n_accepted=s["n_accepted"])
        if s["pending_h"] is not None:
            out["pending_h"] = s["pending_h"]
        return out
    if "desc" not in s:
        s["desc"] = svr.KvDesc(case["heads"], case["kv_heads"], case["dim"], case["page"],
                               window=case.get("window", 0))
        s["batch"] = svr.KvBatch(s["offsets"], s["lens"], s["table"], s["max_rows"])
    if case["op"] == "attention":
        if "ws" not in s:
            s["ws"] = svr.kv_workspace(s["desc"], s["batch"], s["q"].shape[0])
        svr.moe_kv_tree_attention(s["desc"], s["batch"], s["mask"], s["q"], s["cache"], s["out"], ws=s["ws"])
        return s["out"]
    if "kept_batch" not in s:
        s["kept_batch"] = svr.KvBatch(s["kept_offsets"], s["kept_lens"], s["table"], s["max_kept"])
    svr.moe_kv_commit(s["desc"], s["batch"], s["path"], s["n_accepted"], s["caches"], s["kept"])
    for cache, k, v in zip(s["caches"], s["k_out"], s["v_out"]):
        svr.moe_kv_read(s["desc"], s["kept_batch"], cache, k, v)
    return dict(k=s["k_out"], v=s["v_out"], kept=s["kept"])


def run(state):
    if own:
        return _own(state)
    return {"plan": _tree_plan, "attention": _attention, "sample": _sample,
            "commit": _commit}[state["case"]["op"]](state)


def work(case):
    rows, trees, lens = _plan(case)
    T, B, M = sum(rows), len(rows), max(rows)
    if case["op"] == "plan":
        # Parents, offsets and lengths read; masks and positions written.
        return {"bytes": 8 * T + 8 * B + 8 * T * -(-M // 64),
                "flops": sum(len(a) for t in trees for a in _ancestors(t))}
    if case["op"] == "sample":
        V, size = case["vocab"], TYPES[case["dtype"]].itemsize
        # The logits of a path of full length, of each sequence; the draft's probabilities of its last row.
        levels = sum(max(len(a) for a in _ancestors(t)) for t in trees)
        drawn = V * 4 if case["drawn"] else 0
        return {"bytes": levels * V * size + B * (drawn + 8 * M + 8 * case["hidden"]) + 12 * T,
                "flops": 5 * levels * V + B * V * (5 if case["drawn"] else 2)}
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    held = Hk * (D + D // 16)  # bytes of one token in the cache
    if case["op"] == "commit":
        kept = sum(len(p) for p in _kept(case))
        moved = kept - B  # the root stays
        # Tokens read and written; the committed rows read back as 32-bit values.
        return {"bytes": case["layers"] * (2 * moved * held + kept * (held + 8 * Hk * D)) + 12 * B,
                "flops": case["layers"] * kept * 2 * Hk * D}
    size, W = TYPES[case["dtype"]].itemsize, case["window"] or 1 << 30
    seen = [[min(n - r + len(a), W) for a in _ancestors(t)] for r, t, n in zip(rows, trees, lens)]
    held_tokens = sum(min(n, W + r - 1) for r, n in zip(rows, lens))
    return {"bytes": held_tokens * held + 2 * T * Hq * D * size + 8 * T * -(-M // 64),
            "flops": 4 * sum(sum(x) for x in seen) * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    rows, trees, lens = _plan(case)
    if case["op"] == "plan":
        base = (s["lens"].cpu() - torch.tensor(rows)).tolist()
        at = [base[b] + len(a) - 1 for b, t in enumerate(trees) for a in _ancestors(t)]
        return dict(mask=_masks(trees, s["mask"].shape[1]).cuda(), positions=_int32(at))
    if case["op"] == "sample":
        return _exact_sample(s, rows, trees)
    if case["op"] == "commit":
        return _exact_commit(s, rows, lens)
    D, P, W, Hk = case["dim"], case["page"], case["window"], case["kv_heads"]
    G, out, first = case["heads"] // Hk, [], 0
    for b, (r, n) in enumerate(zip(rows, lens)):
        pages = s["cache"][s["table"][b, :-(-n // P)].long()]
        q = s["q"][first:first + r].double()
        first += r
        hidden = torch.ones((r, n), dtype=torch.bool)
        for i, a in enumerate(_ancestors(trees[b])):
            tokens = list(range(max(0, n - r + len(a) - W), n - r)) if W else None
            if W:
                hidden[i, (tokens + [n - r + j for j in a])[-W:]] = False
            else:
                hidden[i, :n - r] = False
                hidden[i, [n - r + j for j in a]] = False
        hidden = hidden.cuda()
        of = torch.empty_like(q)
        for h in range(Hk):
            k, v = _exact_tokens(pages[:, h], D, P, n)
            for i in range(h * G, h * G + G):
                x = (q[:, i] @ k.T / D ** 0.5).masked_fill_(hidden, float("-inf"))
                of[:, i] = torch.softmax(x, -1) @ v
        out.append(of)
    return torch.cat(out)


def _exact_tokens(pages, D, P, n):
    """Keys and values of the first n tokens of one KV head's pages, in 64 bits."""
    half, eighth = P * D // 2, P * D // 32
    both = []
    for c0, s0 in ((0, 2 * half), (half, 2 * half + eighth)):
        byte = pages[:, c0:c0 + half].reshape(-1, D // 2)[:n]
        nib = torch.stack([byte % 16, byte // 16], -1).reshape(-1, D // 32, 32).long()
        mag, sign = nib % 8, 1 - 2 * (nib // 8)
        # A code of exponent e > 0 and fraction f stands for (1 + f / 2) 2^(e-1), of e = 0 for f / 2.
        e, f = mag // 2, mag % 2
        v = torch.where(e > 0, (1 + f / 2).double() * 2.0 ** (e - 1).double(), f / 2) * sign
        scale = pages[:, s0:s0 + eighth].reshape(-1, D // 32, 1)[:n].double()
        both.append((v * 2.0 ** (scale - 127)).reshape(-1, D))
    return both


def _exact_sample(s, rows, trees):
    """Sequence by sequence, from the root, by the definition: a rejected draft's distribution is taken
    off the target's and what is left is normalised."""
    case = s["case"]
    M, first, stop = max(rows), _offsets(rows), []
    tokens, u = s["tokens"].tolist(), s["accept_u"].double().tolist()
    sample_u, temperature = s["sample_u"].double().tolist(), s["temperature"].double().tolist()
    out = dict(accepted=[], path=[], n_accepted=[])
    for b, parents in enumerate(trees):
        node, path, accepted = 0, [0], []
        while True:
            x = s["logits"][first[b] + node].double()
            if temperature[b] > 0:
                p = torch.softmax(x / temperature[b], -1)
            else:
                p = torch.nn.functional.one_hot(x.argmax(), x.shape[0]).double()
            went = None
            for c in [j for j in range(1, rows[b]) if parents[j] == node]:
                t = tokens[first[b] + c]
                px = p[t].item()
                if s["draft_probs"] is None or temperature[b] <= 0:
                    if u[first[b] + c] < px:
                        went = c
                        break
                    if px > 0:
                        p = p.clone()
                        p[t] = 0.0
                else:
                    q = s["draft_probs"][first[b] + node].double()
                    if u[first[b] + c] * q[t].item() < px:
                        went = c
                        break
                    p = (p - q).clamp(min=0.0)
                p = p / p.sum()
            if went is None:
                break
            node = went
            path.append(node)
            accepted.append(tokens[first[b] + node])
        left = p.cumsum(-1)
        accepted.append(int(torch.searchsorted(left, sample_u[b] * left[-1], right=True)))
        stop.append(first[b] + node)
        out["n_accepted"].append(len(path) - 1)
        out["path"].append(path + [-1] * (M - len(path)))
        out["accepted"].append(accepted + [-1] * (M - len(accepted)))
    out = {k: _int32(v) for k, v in out.items()}
    if case["hidden"]:
        out["pending_h"] = s["verify_h"][stop].double()
    return out


def _exact_commit(s, rows, lens):
    case = s["case"]
    D, P, Hk = case["dim"], case["page"], case["kv_heads"]
    out = dict(k=[], v=[])
    kept = [n - r + len(p) for n, r, p in zip(lens, rows, _kept(case))]
    for cache in s["caches"]:
        both = ([], [])
        for b, (r, n, path) in enumerate(zip(rows, lens, _kept(case))):
            lo = (n - r) // P  # the first page that holds new rows
            pages = cache[s["table"][b, lo:-(-n // P)].long()]
            at = [n - r - lo * P + j for j in path]
            heads = [_exact_tokens(pages[:, h], D, P, n - lo * P) for h in range(Hk)]
            for side in (0, 1):
                both[side].append(torch.stack([h[side][at] for h in heads], 1))
        out["k"].append(torch.cat(both[0]))
        out["v"].append(torch.cat(both[1]))
    return dict(out, kept=_int32(kept))
