"""Checks of the 4-bit cache and the log probabilities that need no GPU: the
oracles against closed forms, and every refusal of the C ABI and the binding
(nothing is enqueued: the addresses below are never read)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_verify_router_amd as svr
from speculative_verify_router_amd import _binding as B
from oracle import kv_oracle as ko
from oracle import logprobs_oracle as lo

A = 4096  # an aligned address that no check looks behind


# ---- the oracles -------------------------------------------------------

def test_every_code_value_is_a_fixed_point():
    for e in (-126, -3, 0, 5, 125):
        v = np.concatenate([ko.MAGNITUDES, -ko.MAGNITUDES, ko.MAGNITUDES[::-1], [6] * 8]) * 2.0 ** e
        c, s = ko.block_codes(v)
        assert s == e + 127
        cb = (c[0::2] | c[1::2] << 4)
        assert np.array_equal(ko.vector_values(cb, np.array([s])), v)


def test_no_value_is_off_by_more_than_half_the_widest_step():
    rng = np.random.default_rng(0)
    for _ in range(200):
        x = rng.standard_normal(32) * 10.0 ** rng.uniform(-6, 6)
        c, s = ko.block_codes(x)
        v = ko.vector_values(c[0::2] | c[1::2] << 4, np.array([s]))
        step = np.where(np.abs(v) < 2.0 ** (s - 126), 0.5, np.where(np.abs(v) < 2.0 ** (s - 125), 1, 2))
        assert np.all(np.abs(v - x) <= step / 2 * 2.0 ** (s - 127) * (1 + 1e-12))
        # One exponent less would break that.
        assert np.max(np.abs(x)) > 7 * 2.0 ** (s - 128)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation_of_its_position(interleaved):
    rng = np.random.default_rng(1)
    lay = ko.Layout(1, 1, 64, rotary=64, interleaved=interleaved)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    dots = [ko.head_vector(lay, q, None, f, p + 9) @ ko.head_vector(lay, k, None, f, p) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0], rtol=1e-9)   # the distance alone counts
    assert np.allclose(ko.head_vector(lay, q, None, f, 0), q)
    y = ko.head_vector(lay, q, np.ones(64), f, 3)
    assert math.isclose(np.mean(y * y), 1.0, rel_tol=1e-5)


def test_attention_oracle_on_equal_scores_is_the_mean():
    rng = np.random.default_rng(2)
    lay = ko.Layout(2, 1, 64, 16, window=5)
    cache = rng.integers(0, 256, (2, 1, lay.page_bytes)).astype(np.uint8)
    for p in range(2):
        for part in ko.page_parts(lay, cache[p, 0])[2:]:
            part[:] = 127
    q = np.zeros((3, 2, 64))
    out, lse, *_ = ko.attention(lay, cache, [0, 3], [20], np.array([[1, 0]]), q)
    _, V, _ = ko.stored(lay, cache, np.array([1, 0]), 20, 0)
    for i, place in enumerate((17, 18, 19)):
        assert np.allclose(out[i, 0], V[place - 4:place + 1].mean(0))
        assert math.isclose(lse[i, 1], math.log(5))


def test_logprobs_oracle():
    assert np.allclose(lo.row_logprobs([0, 0, 0, 0]), -math.log(4))
    assert math.isclose(lo.entropy([1, 1, 1]), math.log(3))
    assert lo.entropy([-np.inf, -np.inf]) == 0 and lo.row_logprobs([-np.inf] * 2).tolist() == [-np.inf] * 2
    assert math.isnan(lo.entropy([0, np.nan])) and lo.top_columns([0, np.nan, 3, 3, -np.inf], 5) == [2, 3, 0, 1, 4]
    x = np.random.default_rng(3).standard_normal(5000).round(1)
    assert lo.top_columns(x, 20) == sorted(range(5000), key=lambda c: (-x[c], c))[:20]


# ---- refusals ----------------------------------------------------------

def kv_desc(**kw):
    d = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=64)
    d.update(kw)
    return svr.KvDesc(**d)


def kv_batch(**kw):
    d = dict(n_seqs=2, n_tokens=5, max_rows=4, pages_per_seq=10, q_offsets=A, seq_lens=A, page_table=A)
    d.update(kw)
    return B._KvBatch(*d.values())


BAD_DESC = [
    (dict(head_dim=80), B.ERR_SHAPE), (dict(head_dim=0), B.ERR_SHAPE), (dict(n_heads=7), B.ERR_SHAPE),
    (dict(n_kv_heads=0), B.ERR_SHAPE), (dict(n_heads=0), B.ERR_SHAPE), (dict(n_heads=2048), B.ERR_SHAPE),
    (dict(page_size=8), B.ERR_SHAPE), (dict(page_size=48), B.ERR_SHAPE), (dict(page_size=2048), B.ERR_SHAPE),
    (dict(window=-1), B.ERR_SHAPE), (dict(rotary_dims=8), B.ERR_SHAPE), (dict(rotary_dims=144), B.ERR_SHAPE),
    (dict(rotary_dims=-16), B.ERR_SHAPE), (dict(scale=-1.0), B.ERR_ARG), (dict(scale=math.nan), B.ERR_ARG),
    (dict(scale=math.inf), B.ERR_ARG), (dict(norm_eps=-1e-6), B.ERR_ARG), (dict(norm_eps=math.nan), B.ERR_ARG),
]
BAD_BATCH = [
    (dict(n_seqs=-1), B.ERR_SHAPE), (dict(n_seqs=65537), B.ERR_SHAPE), (dict(n_tokens=-1), B.ERR_SHAPE),
    (dict(n_tokens=2 ** 20 + 1), B.ERR_SHAPE), (dict(max_rows=-1), B.ERR_SHAPE),
    (dict(pages_per_seq=0), B.ERR_SHAPE), (dict(pages_per_seq=2 ** 14 + 1), B.ERR_SHAPE),
]
BAD_ARRAYS = [
    (dict(q_offsets=None), B.ERR_NULL), (dict(seq_lens=None), B.ERR_NULL), (dict(page_table=None), B.ERR_NULL),
    (dict(q_offsets=A + 2), B.ERR_ARG), (dict(page_table=A + 1), B.ERR_ARG),
]


def append_status(desc=None, batch=None, **kw):
    a = dict(dtype=B.BF16, q=A, qs=1024, k=A, ks=256, v=A, vs=256, qn=A, kn=A, f=A, pos=A, cache=A,
             n_pages=4, q_out=A, stream=None)
    a.update(kw)
    return svr.lib().moe_kv_append((desc or kv_desc()).c(), batch or kv_batch(), *a.values())


def attention_status(desc=None, batch=None, **kw):
    a = dict(dtype=B.BF16, q=A, qs=1024, cache=A, n_pages=4, out=A, lse=A, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return svr.lib().moe_kv_attention((desc or kv_desc()).c(), batch or kv_batch(), *a.values())


def read_status(desc=None, batch=None, **kw):
    a = dict(cache=A, n_pages=4, k=A, v=A, stream=None)
    a.update(kw)
    return svr.lib().moe_kv_read((desc or kv_desc()).c(), batch or kv_batch(), *a.values())


@pytest.mark.parametrize("call", [append_status, attention_status, read_status])
def test_kv_calls_refuse_bad_descriptions(call):
    for kw, status in BAD_DESC:
        assert call(desc=kv_desc(**kw)) == status, kw
    for kw, status in BAD_BATCH + BAD_ARRAYS:
        assert call(batch=kv_batch(**kw)) == status, kw
    d = kv_desc().c()
    d.flags = 2
    f = {append_status: "moe_kv_append", attention_status: "moe_kv_attention", read_status: "moe_kv_read"}[call]
    n = len(getattr(svr.lib(), f).argtypes)
    assert getattr(svr.lib(), f)(d, kv_batch(), *([0] * (n - 2))) == B.ERR_ARG
    assert getattr(svr.lib(), f)(None, kv_batch(), *([0] * (n - 2))) == B.ERR_NULL
    assert getattr(svr.lib(), f)(kv_desc().c(), None, *([0] * (n - 2))) == B.ERR_NULL
    assert call(n_pages=0) == B.ERR_SHAPE and call(n_pages=-4) == B.ERR_SHAPE
    assert call(cache=None) == B.ERR_NULL and call(cache=A + 8) == B.ERR_ARG


def test_append_refusals():
    for kw, status in [
        (dict(dtype=B.Q8_0), B.ERR_DTYPE), (dict(dtype=99), B.ERR_DTYPE), (dict(k=None), B.ERR_NULL),
        (dict(v=None), B.ERR_NULL), (dict(q=None), B.ERR_NULL), (dict(q_out=None), B.ERR_NULL),
        (dict(qs=1023), B.ERR_SHAPE), (dict(ks=255), B.ERR_SHAPE), (dict(vs=-256), B.ERR_SHAPE),
        (dict(q=A + 1), B.ERR_ARG), (dict(dtype=B.F32, k=A + 2), B.ERR_ARG), (dict(q_out=A + 1), B.ERR_ARG),
        (dict(qn=A + 2), B.ERR_ARG), (dict(pos=A + 1), B.ERR_ARG),
    ]:
        assert append_status(**kw) == status, kw
    assert append_status(desc=kv_desc(rotary_dims=64), f=None) == B.ERR_NULL


def test_attention_refusals():
    for kw, status in [
        (dict(dtype=B.Q4_K), B.ERR_DTYPE), (dict(q=None), B.ERR_NULL), (dict(out=None), B.ERR_NULL),
        (dict(qs=1000), B.ERR_SHAPE), (dict(q=A + 1), B.ERR_ARG), (dict(out=A + 1), B.ERR_ARG),
        (dict(lse=A + 2), B.ERR_ARG), (dict(ws=None), B.ERR_NULL), (dict(ws=A + 128), B.ERR_ARG),
        (dict(ws_bytes=100), B.ERR_WORKSPACE),
    ]:
        assert attention_status(**kw) == status, kw
    out = ctypes.c_size_t()
    f = svr.lib().moe_kv_attention_workspace_bytes
    assert f(kv_desc().c(), kv_batch(), None) == B.ERR_NULL
    assert f(kv_desc(head_dim=96).c(), kv_batch(), ctypes.byref(out)) == B.ERR_SHAPE
    assert f(kv_desc().c(), kv_batch(q_offsets=None), ctypes.byref(out)) == B.OK


def test_read_refuses_no_output():
    assert read_status(k=None, v=None) == B.ERR_NULL
    assert read_status(k=A + 2) == B.ERR_ARG


def test_empty_batches_enqueue_nothing():
    for b in (kv_batch(n_tokens=0), kv_batch(n_seqs=0, q_offsets=None, seq_lens=None, page_table=None)):
        assert append_status(batch=b) == B.OK
        assert attention_status(batch=b) == B.OK
        assert read_status(batch=b) == B.OK
    assert attention_status(batch=kv_batch(max_rows=0)) == B.OK


def test_cache_bytes():
    assert svr.moe_kv_cache_bytes(kv_desc(), 3) == 3 * 2 * 64 * (128 + 8)
    assert svr.moe_kv_cache_bytes(kv_desc(head_dim=256, page_size=1024, n_kv_heads=8), 100000) == 100000 * 8 * 1024 * 272
    for n in (0, -1, 2 ** 31):
        with pytest.raises(svr.MoeError) as e:
            svr.moe_kv_cache_bytes(kv_desc(), n)
        assert e.value.status == B.ERR_SHAPE


def logprobs_status(**kw):
    a = dict(x=A, dtype=B.F32, rows=4, V=1000, stride=1000, targets=A, lp=A, h=A, k=5, ids=A, tl=A, ws=A,
             ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return svr.lib().moe_logprobs(*a.values())


def test_logprobs_refusals():
    for kw, status in [
        (dict(rows=-1), B.ERR_SHAPE), (dict(rows=2 ** 20 + 1), B.ERR_SHAPE), (dict(V=0), B.ERR_SHAPE),
        (dict(V=2 ** 30 + 1, stride=2 ** 31), B.ERR_SHAPE), (dict(stride=999), B.ERR_SHAPE),
        (dict(k=-1), B.ERR_SHAPE), (dict(k=65), B.ERR_SHAPE), (dict(V=3, k=4), B.ERR_SHAPE),
        (dict(dtype=B.Q8_0), B.ERR_DTYPE), (dict(x=None), B.ERR_NULL), (dict(ws=None), B.ERR_NULL),
        (dict(targets=None), B.ERR_NULL), (dict(lp=None), B.ERR_NULL), (dict(ws_bytes=100), B.ERR_WORKSPACE),
        (dict(ws=A + 64), B.ERR_ARG), (dict(x=A + 2), B.ERR_ARG), (dict(h=A + 1), B.ERR_ARG),
        (dict(ids=A + 2), B.ERR_ARG), (dict(tl=A + 2), B.ERR_ARG),
    ]:
        assert logprobs_status(**kw) == status, kw
    assert logprobs_status(rows=0) == B.OK
    assert svr.lib().moe_logprobs_workspace_bytes(4, 1000, 5, None) == B.ERR_NULL
    for a in ((-1, 1000, 0), (4, 0, 0), (4, 1000, 65), (4, 3, 4)):
        with pytest.raises(svr.MoeError) as e:
            svr.moe_logprobs_workspace_bytes(*a)
        assert e.value.status == B.ERR_SHAPE


def test_logprobs_workspace_serves_every_smaller_batch():
    for V, k in ((131072, 20), (5000, 64), (1000, 0)):
        most = svr.moe_logprobs_workspace_bytes(600, V, k)
        for rows in (1, 2, 3, 7, 64, 100, 511, 512, 513, 600):
            assert svr.moe_logprobs_workspace_bytes(rows, V, k) <= most


def test_the_binding_refuses_what_it_cannot_pass_on():
    d = kv_desc()
    batch = svr.KvBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                        torch.zeros((1, 4), dtype=torch.int32), 1)
    cache = torch.zeros((4, 2, d.page_bytes), dtype=torch.uint8)
    q, kv = torch.zeros((1, 8, 128)), torch.zeros((1, 2, 128))
    with pytest.raises(ValueError, match="device tensor"):
        svr.moe_kv_append(d, batch, q, kv, kv, cache, torch.zeros_like(q))
    with pytest.raises(ValueError, match="q: expected shape"):
        svr.moe_kv_append(d, batch, q[:, :4], kv, kv, cache, torch.zeros_like(q))
    with pytest.raises(ValueError, match="v: expected torch.float32"):
        svr.moe_kv_append(d, batch, q, kv, kv.half(), cache, torch.zeros_like(q))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        svr.moe_kv_append(d, batch, None, kv.double(), kv.double(), cache, None)
    with pytest.raises(ValueError, match="k: expected whole rows"):
        svr.moe_kv_append(d, batch, None, torch.zeros((1, 128, 2)).transpose(1, 2), kv, cache, None)
    with pytest.raises(ValueError, match="cache: expected shape"):
        svr.moe_kv_append(d, batch, None, kv, kv, cache[:, :1], None)
    with pytest.raises(ValueError, match="inv_freq: expected shape"):
        svr.moe_kv_append(kv_desc(rotary_dims=64), batch, None, kv, kv, cache, None, inv_freq=torch.zeros(16))
    with pytest.raises(ValueError, match="seq_lens: expected shape"):
        svr.KvBatch(batch.q_offsets, torch.zeros(2, dtype=torch.int32), batch.page_table, 1)
    with pytest.raises(ValueError, match="out: expected shape"):
        svr.moe_kv_attention(d, batch, q, cache, q[:, :4], ws=cache.view(-1))
    with pytest.raises(ValueError, match="k_out or v_out"):
        svr.moe_kv_read(d, batch, cache, None, None)
    x = torch.zeros((2, 10))
    with pytest.raises(ValueError, match="vocabulary"):
        svr.moe_logprobs(x[0], None, None, ws=cache.view(-1))
    with pytest.raises(ValueError, match="whole rows"):
        svr.moe_logprobs(x.T, None, None, ws=cache.view(-1))
    with pytest.raises(ValueError, match="targets: expected torch.int32"):
        svr.moe_logprobs(x, torch.zeros(2, dtype=torch.int64), torch.zeros(2), ws=cache.view(-1))
    with pytest.raises(ValueError, match="top_logprobs: expected shape"):
        svr.moe_logprobs(x, None, None, None, torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 4)),
                         ws=cache.view(-1))
    with pytest.raises(ValueError, match="device tensor"):
        svr.moe_logprobs(x, None, None, ws=cache.view(-1))


def test_the_binding_refuses_numbers_that_ctypes_would_cut_off():
    with pytest.raises(ValueError, match="window"):
        svr.KvDesc(4, 2, 64, window=2 ** 32 + 5)
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_rows"):
        svr.KvBatch(z, z[:1], z[None], 2 ** 32 + 1)


def test_the_binding_refuses_a_batch_on_another_device():
    """Its addresses would be read by the wrong device."""
    d = svr.KvDesc(4, 2, 64, 16)
    z = torch.zeros(2, dtype=torch.int32)
    batch = svr.KvBatch(z, z[:1], z[None, :1], 1)
    m = dict(device="meta")
    q, k = torch.empty((1, 4, 64), **m), torch.empty((1, 2, 64), **m)
    cache = torch.empty((1, 2, d.page_bytes), dtype=torch.uint8, **m)
    f = torch.empty((1, 2, 64), **m)
    ws = torch.empty(0, dtype=torch.uint8, **m)
    for call in (lambda: svr.moe_kv_append(d, batch, q, k, k, cache, q),
                 lambda: svr.moe_kv_attention(d, batch, q, cache, q, ws=ws),
                 lambda: svr.moe_kv_read(d, batch, cache, f, f)):
        with pytest.raises(ValueError, match="batch: expected tensors on meta"):
            call()


@pytest.mark.parametrize("seqs,rows,max_rows", [(0, 0, 1), (0, 3, 1), (2, 0, 1), (2, 5, 0), (1, 5, 0)])
def test_attention_of_nothing_needs_no_workspace(seqs, rows, max_rows):
    i32 = dict(dtype=torch.int32)
    batch = svr.KvBatch(torch.zeros(seqs + 1, **i32), torch.zeros(seqs, **i32),
                        torch.zeros((seqs, 9), **i32), max_rows)
    assert svr.moe_kv_attention_workspace_bytes(kv_desc(), batch, rows) == 0


def test_more_work_than_a_launch_can_take_is_refused():
    """2^32 threads or more: a launch would be refused, after the checks."""
    wide = dict(n_heads=1024, n_kv_heads=1024, head_dim=256)
    many = kv_batch(n_seqs=65536, n_tokens=65536, max_rows=1)
    assert 65536 * 1024 * 256 >= 2 ** 32
    assert attention_status(desc=kv_desc(**wide), batch=many, qs=1024 * 256) == B.ERR_SHAPE
    long = kv_batch(n_seqs=1, n_tokens=2 ** 20, max_rows=2 ** 20)
    assert 2 ** 20 * 1024 // 32 * 256 >= 2 ** 32
    assert attention_status(desc=kv_desc(n_heads=1024, n_kv_heads=64), batch=long, qs=1024 * 128) == B.ERR_SHAPE
    assert read_status(desc=kv_desc(**wide), batch=long) == B.ERR_SHAPE


@pytest.mark.parametrize("heads,kv_heads,dim", [(64, 4, 192), (32, 8, 128), (8, 8, 64), (16, 1, 256)])
def test_sequences_of_a_long_table_can_be_cut_however_many_there_are(heads, kv_heads, dim):
    """One long sequence among short ones must not be walked by a workgroup a head alone.  What parts need does not
    go by the rows or sequences."""
    d = kv_desc(n_heads=heads, n_kv_heads=kv_heads, head_dim=dim)
    for seqs in (1, 2, 64, 65, 96, 97, 128, 200, 512, 1024, 1025, 4000):
        out = ctypes.c_size_t()
        b = kv_batch(n_seqs=seqs, n_tokens=seqs, max_rows=1, pages_per_seq=1000)
        assert svr.lib().moe_kv_attention_workspace_bytes(d.c(), b, ctypes.byref(out)) == B.OK
        assert 16384 < out.value < 2 ** 26, seqs


@pytest.mark.parametrize("heads,kv_heads,dim,window", [(64, 4, 192, 0), (32, 8, 128, 512), (8, 8, 64, 0), (1024, 1024, 256, 0)])
def test_attention_workspace_serves_every_smaller_batch(heads, kv_heads, dim, window):
    """Fewer rows are cut into more parts: a size that went by one batch alone would be too little for others."""
    d = kv_desc(n_heads=heads, n_kv_heads=kv_heads, head_dim=dim, window=window)

    def need(seqs, rows, max_rows, pages):
        out = ctypes.c_size_t()
        b = kv_batch(n_seqs=seqs, n_tokens=rows, max_rows=max_rows, pages_per_seq=pages)
        assert svr.lib().moe_kv_attention_workspace_bytes(d.c(), b, ctypes.byref(out)) == B.OK
        return out.value

    most = need(256, 4096, 2048, 1000)
    assert most < 60e6
    for seqs in (1, 2, 3, 64, 100, 256):
        for rows in (1, 4, 64, 512, 4096):
            for max_rows in (1, 4, 33, 2048):
                for pages in (1, 7, 1000):
                    assert need(seqs, rows, max_rows, pages) <= most


def test_the_binding_refuses_a_scale_that_is_none_in_32_bits():
    """A scale of zero stands for 1/sqrt(head_dim)."""
    for scale in (1e-50, 5e-324):
        with pytest.raises(ValueError, match="scale"):
            svr.KvDesc(4, 2, 64, scale=scale)
    assert svr.KvDesc(4, 2, 64, scale=1e-38).c().scale > 0 and svr.KvDesc(4, 2, 64).c().scale == 0


def test_the_binding_refuses_sizes_that_ctypes_would_cut_off():
    z = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: svr.moe_logprobs_workspace_bytes(2 ** 32 + 4, 1000),
                 lambda: svr.moe_logprobs_workspace_bytes(4, 2 ** 64 + 1000),
                 lambda: svr.moe_logprobs_workspace_bytes(4, 1000, 2 ** 32),
                 lambda: svr.moe_kv_cache_bytes(kv_desc(), 2 ** 64 + 1),
                 lambda: svr.moe_kv_attention_workspace_bytes(kv_desc(), svr.KvBatch(z, z[:1], z[None], 1), 2 ** 32 + 1)):
        with pytest.raises((ValueError, svr.MoeError)):
            call()
