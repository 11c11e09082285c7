"""Cases of the verify step's operators around the MoE layer, and their plain forms.

Three operators: appending the queries, keys and values of a batch to a paged
4-bit cache (head norms and position rotation on the way), attention over that
cache, and log probabilities with entropy and top alternatives.  Each case is a
dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` makes one
pass: with ``own`` the framework's calls, without it elementary torch
operations in 32 bits (64 where a border or a far angle needs it).
"""

from __future__ import annotations

import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# Values of the 4-bit codes (E2M1): bit 3 is the sign.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# The most a drawn case may cost: what the largest listed ones cost.
MOST_APPEND_ELEMENTS = 2048 * (64 + 2 * 4) * 192
MOST_PAIRS = 512 * 64 * 16384 * 192      # query rows x heads x visible tokens x head size
MOST_CACHE = 60000 * 4 * 192             # tokens x KV heads x head size
MOST_LOGITS = 512 * 131072


def listed():
    a = dict(op="append", interleaved=False, norm=True)
    t = dict(op="attention", window=0, ragged=False)
    p = dict(op="logprobs", masked=False)
    return [
        # One verify batch (the last accepted token and three drafts) of the Step-5 head layout.
        dict(a, name="append_verify_m4", dtype="bf16", heads=64, kv_heads=4, dim=192, page=64,
             rotary=64, seqs=1, rows=4, length=60000, ragged=False),
        # A decode step of many sequences, small pages, pairs of neighbours rotated.
        dict(a, name="append_decode_b61", dtype="f16", heads=32, kv_heads=8, dim=128, page=16,
             rotary=128, seqs=61, rows=1, length=9000, ragged=True, interleaved=True),
        # A prefill micro-batch of 512 tokens in the layer's own 32-bit activations.
        dict(a, name="append_prefill_512", dtype="f32", heads=64, kv_heads=4, dim=192, page=64,
             rotary=64, seqs=1, rows=512, length=8192, ragged=False),
        # The largest prefill chunk, two prompts of different lengths.
        dict(a, name="append_prefill_2048", dtype="bf16", heads=64, kv_heads=4, dim=192, page=128,
             rotary=192, seqs=2, rows=1024, length=16384, ragged=True),
        # Single-token decode on a short cache: latency counts.
        dict(t, name="attention_m1_short", dtype="bf16", heads=64, kv_heads=4, dim=192, page=64,
             seqs=1, rows=1, length=777),
        # The verify batch on a prompt of 60000 tokens.
        dict(t, name="attention_m4_60000", dtype="bf16", heads=64, kv_heads=4, dim=192, page=64,
             seqs=1, rows=4, length=60000),
        # Many sequences of uneven lengths, up to four rows each.
        dict(t, name="attention_b29_ragged", dtype="f16", heads=32, kv_heads=8, dim=128, page=16,
             seqs=29, rows=4, length=5000, ragged=True),
        # A sliding-window layer in 32-bit activations.
        dict(t, name="attention_window_512", dtype="f32", heads=64, kv_heads=4, dim=192, page=64,
             seqs=8, rows=4, length=6001, ragged=True, window=512),
        # A prefill micro-batch at the end of a long prompt.
        dict(t, name="attention_prefill_512", dtype="bf16", heads=64, kv_heads=4, dim=192, page=64,
             seqs=1, rows=512, length=16384),
        # One sampled token, no alternatives asked for.
        dict(p, name="logprobs_m1", dtype="f32", rows=1, vocab=131072, top=0),
        # The verify batch with twenty alternatives, under a grammar's mask of -inf.
        dict(p, name="logprobs_m4_top20", dtype="f32", rows=4, vocab=131072, top=20, masked=True),
        # Log probabilities of a whole prefill micro-batch, 16-bit logits.
        dict(p, name="logprobs_prompt_512", dtype="bf16", rows=512, vocab=131072, top=5),
    ]


def _log_int(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "logprobs"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "logprobs":
        vocab = _log_int(rng, 1000, 262144)
        rows = _log_int(rng, 1, max(1, min(2048, MOST_LOGITS // 2 // vocab)))
        return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, top=rng.choice([0, 1, 5, 8, 20, 32]),
                    masked=rng.random() < 0.3)
    dim = rng.choice([64, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    if op == "append":
        most = max(1, MOST_APPEND_ELEMENTS // 2 // ((heads + 2 * kv_heads) * dim))
        tokens = _log_int(rng, 1, min(2048, most))
        seqs = _log_int(rng, 1, min(64, tokens))
        rows = max(1, tokens // seqs)
        return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    rotary=rng.choice([r for r in (0, 32, 64, dim) if r <= dim]), seqs=seqs,
                    rows=rows, length=rows + _log_int(rng, 1, 20000), ragged=ragged,
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.7)
    seqs = _log_int(rng, 1, 48)
    most = max(64, MOST_CACHE // (seqs * kv_heads * dim))
    length = _log_int(rng, 1, min(60000, most))
    if dtype == "f32":
        length = min(length, 20000)
    rows = rng.choice([1, 1, 2, 3, 4, _log_int(rng, 1, 512)])
    rows = max(1, min(rows, length, MOST_PAIRS // (4 * seqs * heads * length * dim)))
    return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                window=rng.choice([0, 0, 0, 512, 100]), seqs=seqs, rows=rows, length=length,
                ragged=ragged)


def _plan(case):
    """Rows and lengths (with the new rows) of every sequence: the case's own, whatever the seed."""
    n, rows, length = case["seqs"], case["rows"], case["length"]
    if not case["ragged"]:
        return [rows] * n, [length] * n
    rng = random.Random(n * 1000003 + rows * 8191 + length)
    r = [rows] + [rng.randint(1, rows) for _ in range(n - 1)]
    return r, [length] + [rng.randint(max(x, length // 16, 1), length) for x in r[1:]]


def _page_bytes(dim, page):
    """Codes of keys, codes of values (4 bits each), scales of keys, scales of values (a byte for 32)."""
    return page * (dim + dim // 16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "logprobs":
        N, V = case["rows"], case["vocab"]
        x = normal(N, V).mul_(2.5)
        # A few likely tokens on top of the bulk, as a trained model gives.
        likely = torch.randint(0, V, (N, 8), generator=g, device="cuda")
        x.scatter_add_(1, likely, 8.0 + 3.0 * normal(N, 8))
        targets = torch.where(torch.rand(N, generator=g, device="cuda") < 0.7, likely[:, 0],
                              torch.randint(0, V, (N,), generator=g, device="cuda"))
        if case["masked"]:
            keep = torch.rand((N, V), generator=g, device="cuda") < 0.1
            keep.scatter_(1, targets[:, None], True)
            x.masked_fill_(~keep, float("-inf"))
        k = case["top"]
        f32 = dict(dtype=torch.float32, device="cuda")
        return dict(case=case, logits=x.to(dt), targets=targets.int(),
                    logprobs=torch.empty(N, **f32), entropy=torch.empty(N, **f32),
                    top_ids=torch.empty((N, k), dtype=torch.int32, device="cuda"),
                    top_logprobs=torch.empty((N, k), **f32))

    Hq, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    rows, lens = _plan(case)
    T, width = sum(rows), -(-max(lens) // P)
    used = [-(-x // P) for x in lens]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    take = torch.tensor([[sum(used[:b]) + min(i, used[b] - 1) for i in range(width)]
                         for b in range(len(lens))], device="cuda")
    offsets = torch.tensor([sum(rows[:b]) for b in range(len(rows) + 1)], dtype=torch.int32)
    s = dict(case=case, offsets=offsets.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
             table=order[take], max_rows=max(rows))
    if case["op"] == "append":
        R = case["rotary"]
        qkv = normal(T, (Hq + 2 * Hk) * D).to(dt)  # one row of the fused projection a token
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
        s["q_norm"] = 1.0 + 0.1 * normal(D) if case["norm"] else None
        s["k_norm"] = 1.0 + 0.1 * normal(D) if case["norm"] else None
        s["inv_freq"] = None
        if R:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()
        s["cache"] = torch.zeros((n_pages, Hk, _page_bytes(D, P)), dtype=torch.uint8, device="cuda")
        s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((T, Hk, D), dtype=torch.float32, device="cuda")
        s["v_out"] = torch.empty((T, Hk, D), dtype=torch.float32, device="cuda")
        return s
    s["q"] = normal(T, Hq, D).to(dt)
    codes, scales = _quantise(normal(n_pages, 2, Hk, P, D))
    packed = (codes[..., 0::2] | codes[..., 1::2] << 4).transpose(1, 2).reshape(n_pages, Hk, -1)
    scales = scales.transpose(1, 2).reshape(n_pages, Hk, -1)
    s["cache"] = torch.cat([packed, scales], 2).contiguous()
    s["out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    return s


def _quantise(x):
    """4-bit codes and scale bytes of blocks of 32 along the last axis: the scale is the least power
    of two with max|x| <= 7 of it, the code the nearest of E2M1, the even one between two."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 3, e - 2).clamp(-126, 125)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
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
    n, Hk, _ = cache.shape
    c, s = P * D // 2, P * D // 32
    k, v, ks, vs = cache.split([c, c, s, s], 2)
    return (k.unflatten(2, (P, D // 2)), v.unflatten(2, (P, D // 2)),
            ks.unflatten(2, (P, D // 32)), vs.unflatten(2, (P, D // 32)))


def _append(s):
    case = s["case"]
    D, P, R = case["dim"], case["page"], case["rotary"]
    T = s["q"].shape[0]
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["offsets"].long(), i, right=True) - 1
    at = (s["lens"][b] - s["offsets"][b + 1] + i).long()  # the token's place in its sequence

    def normed(x, w):
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w

    def rotated(x):
        if not R:
            return x
        angle = at[:, None] * s["inv_freq"].double()
        cos, sin = angle.cos()[:, None].to(x.dtype), angle.sin()[:, None].to(x.dtype)
        y = x.clone()
        if case["interleaved"]:
            p, n = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = p * cos - n * sin, n * cos + p * sin
        else:
            p, n = x[..., :R // 2], x[..., R // 2:R]
            y[..., :R // 2], y[..., R // 2:R] = p * cos - n * sin, n * cos + p * sin
        return y

    q = rotated(normed(s["q"].float(), s["q_norm"]))
    # Codes are whole numbers: in 64 bits a value next to a border falls on its own side.
    k = rotated(normed(s["k"].double(), s["k_norm"]))
    kc, ks = _quantise(k)
    vc, vs = _quantise(s["v"].float())
    pages, o = s["table"][b, at // P].long(), at % P
    for part, new in zip(_parts(s["cache"], D, P), (kc[..., 0::2] | kc[..., 1::2] << 4,
                                                    vc[..., 0::2] | vc[..., 1::2] << 4, ks, vs)):
        part[pages, :, o] = new
    return dict(q=q.to(s["q"].dtype), k=_values(kc, ks), v=_values(vc, vs))


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

    t = torch.arange(kc.shape[1], device="cuda")
    at = s["lens"][:, None] - rows[:, None] + j  # place of each row
    see = (t <= at[..., None]) & (t < s["lens"][:, None, None])
    if W:
        see &= t > at[..., None] - W
    see = see[:, None, :, None].expand(B, 1, R, Hq // Hk, -1).reshape(B, 1, R * (Hq // Hk), -1)
    x = (q @ wide(kc, ks).transpose(2, 3)).mul_(D ** -0.5).masked_fill_(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = x.sub_(m.masked_fill(m == float("-inf"), 0.0)).exp_()
    o = (e @ wide(vc, vs)) / e.sum(-1, keepdim=True).clamp_min(1e-37)
    o = o.view(B, Hk, R, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D)
    return o[j < rows[:, None]].to(s["q"].dtype)


def _logprobs(s):
    x = s["logits"].float()
    N, V = x.shape
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = d.exp()
    z = e.sum(-1)
    lse = z.log()
    lp = d.gather(1, s["targets"][:, None].long())[:, 0] - lse
    h = lse - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(-1) / z
    k = s["case"]["top"]
    if not k:
        return dict(logprobs=lp, entropy=h)
    # Order by value, equal ones by the lower index: one 64-bit key of both.
    u = (x + 0.0).view(torch.int32).long()
    u = torch.where(u < 0, -2 ** 31 - u, u)
    key = u * 2 ** 32 + (V - 1 - torch.arange(V, device="cuda"))
    ids = V - 1 - (key.topk(k, 1).values & (2 ** 32 - 1))
    return dict(logprobs=lp, entropy=h, top_ids=ids.int(), top_logprobs=d.gather(1, ids) - lse[:, None])


def _own(s):
    import speculative_verify_router_amd as svr
    case = s["case"]
    if case["op"] == "logprobs":
        if "ws" not in s:
            s["ws"] = svr.logprobs_workspace(case["rows"], case["vocab"], case["top"])
        k = case["top"]
        out = dict(logprobs=s["logprobs"], entropy=s["entropy"])
        if k:
            out |= dict(top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
        svr.moe_logprobs(s["logits"], s["targets"], ws=s["ws"], **out)
        return out
    if "desc" not in s:
        s["desc"] = svr.KvDesc(case["heads"], case["kv_heads"], case["dim"], case["page"],
                               rotary_dims=case.get("rotary", 0),
                               rotary_interleaved=case.get("interleaved", False),
                               window=case.get("window", 0))
        s["batch"] = svr.KvBatch(s["offsets"], s["lens"], s["table"], s["max_rows"])
    if case["op"] == "append":
        svr.moe_kv_append(s["desc"], s["batch"], s["q"], s["k"], s["v"], s["cache"], s["q_out"],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], inv_freq=s["inv_freq"])
        svr.moe_kv_read(s["desc"], s["batch"], s["cache"], s["k_out"], s["v_out"])
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    if "ws" not in s:
        s["ws"] = svr.kv_workspace(s["desc"], s["batch"], s["q"].shape[0])
    svr.moe_kv_attention(s["desc"], s["batch"], s["q"], s["cache"], s["out"], ws=s["ws"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attention": _attention, "logprobs": _logprobs}[state["case"]["op"]](state)


def work(case):
    size = TYPES[case["dtype"]].itemsize
    if case["op"] == "logprobs":
        N, V, k = case["rows"], case["vocab"], case["top"]
        return {"bytes": N * (V * size + 12 + 8 * k), "flops": 5 * N * V}
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    rows, lens = _plan(case)
    T = sum(rows)
    held = Hk * (D + D // 16)  # bytes of one token in the cache
    if case["op"] == "append":
        # q, k, v read; q and the cache written; the appended values read back as 32-bit ones.
        return {"bytes": T * ((2 * Hq + 2 * Hk) * D * size + 2 * held + 2 * Hk * D * 4),
                "flops": T * (Hq + 2 * Hk) * D * 10}
    W = case["window"] or 1 << 30
    seen = [min(n, r - 1 + W) for r, n in zip(rows, lens)]
    pairs = sum(min(n - r + i + 1, W) for r, n in zip(rows, lens) for i in range(r))
    return {"bytes": sum(seen) * held + 2 * T * Hq * D * size, "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    rows, lens = _plan(case)
    if case["op"] == "append":
        return _exact_append(s, rows, lens)
    D, P, W, Hk = case["dim"], case["page"], case["window"], case["kv_heads"]
    G, out, first = case["heads"] // Hk, [], 0
    for b, (r, n) in enumerate(zip(rows, lens)):
        pages = s["cache"][s["table"][b, :-(-n // P)].long()]
        q = s["q"][first:first + r].double()
        first += r
        here = torch.arange(n - r, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")
        hidden = (t > here) | (t + (W or n + 1) <= here)
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


def _exact_append(s, rows, lens):
    case = s["case"]
    R = case["rotary"]
    at = torch.cat([torch.arange(n - r, n) for r, n in zip(rows, lens)]).cuda()

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
        if R:
            a = at[:, None, None].double() * s["inv_freq"].double()
            spin = torch.complex(a.cos(), a.sin())
            if case["interleaved"]:
                z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], -1, 2).contiguous()) * spin
                x = torch.cat([torch.view_as_real(z).flatten(-2), x[..., R:]], -1)
            else:
                z = torch.complex(*x[..., :R].chunk(2, -1)) * spin
                x = torch.cat([z.real, z.imag, x[..., R:]], -1)
        return x

    def stored(x):
        b = x.double().reshape(*x.shape[:2], -1, 32)
        top = b.abs().amax(-1, keepdim=True)
        # The least whole e with top / 7 <= 2^e; log2 near a whole number is put right by the test.
        e = torch.ceil(torch.log2(top / 7).clamp(-200, 200)).clamp(-126, 125)
        e = torch.where(top > 7 * 2.0 ** e, e + 1, e)
        e = torch.where(top <= 7 * 2.0 ** (e - 1), e - 1, e).clamp(-126, 125)
        t = b / 2.0 ** e
        step = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0)).double()
        return ((t / step).round() * step).clamp(-6, 6).mul(2.0 ** e).reshape(x.shape)

    return dict(q=turned(s["q"], s["q_norm"]), k=stored(turned(s["k"], s["k_norm"])), v=stored(s["v"]))


def _exact_logprobs(s):
    x = s["logits"].double()
    lp = torch.log_softmax(x, -1)
    out = dict(logprobs=lp[torch.arange(len(x)), s["targets"].long()],
               entropy=torch.special.entr(lp.exp()).sum(-1))
    if s["case"]["top"]:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :s["case"]["top"]]
        out |= dict(top_ids=order.int(), top_logprobs=lp.gather(1, order))
    return out
