"""ctypes binding of the C ABI in include/*.h.

Argument marshalling only: torch tensors are checked for device, dtype and
contiguity and passed as raw device pointers; the HIP stream is torch's
current stream.  Every step of the layer runs in the HIP library; there is
no fallback, so a missing library raises.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Sequence

import torch  # load torch first: the library then binds to torch's HIP runtime

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libsvr_moe.so")

F32, Q8_0, Q4_K, Q2_K, Q3_K, Q6_K = 0, 1, 2, 3, 4, 5
_DTYPES = {"f32": F32, "q8_0": Q8_0, "q4_k": Q4_K, "q2_k": Q2_K, "q3_k": Q3_K, "q6_k": Q6_K}

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_WORKSPACE, ERR_LAUNCH, ERR_ARG = range(7)


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({strerror(status)})")
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("shared_ffn", ctypes.c_int32), ("expert_type", ctypes.c_int32),
                ("shared_type", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("down_type", ctypes.c_int32)]


class _Weights(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("shared_gate", ctypes.c_void_p),
                ("shared_up", ctypes.c_void_p), ("shared_down", ctypes.c_void_p)]


class _KvDesc(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("window", ctypes.c_int32), ("rotary_dims", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("scale", ctypes.c_float), ("norm_eps", ctypes.c_float)]


class _KvBatch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32),
                ("q_offsets", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


@dataclasses.dataclass(frozen=True)
class LayerDesc:
    hidden: int
    n_experts: int
    top_k: int
    ffn: int
    shared_ffn: int = 0
    expert_type: str = "q4_k"
    shared_type: str = "q8_0"
    down_type: Optional[str] = None  # routed down; None: expert_type

    def c(self) -> _Desc:
        return _Desc(self.hidden, self.n_experts, self.top_k, self.ffn, self.shared_ffn,
                     _DTYPES[self.expert_type], _DTYPES[self.shared_type], 0,
                     _DTYPES[self.down_type] if self.down_type else 0)


@dataclasses.dataclass
class LayerWeights:
    """Device tensors of one layer (uint8 for quantised tensors)."""
    router: torch.Tensor
    gate: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor
    shared_gate: Optional[torch.Tensor] = None
    shared_up: Optional[torch.Tensor] = None
    shared_down: Optional[torch.Tensor] = None

    def c(self) -> _Weights:
        p = lambda t: None if t is None else _ptr(t, None)  # noqa: E731
        return _Weights(_ptr(self.router, torch.float32), p(self.gate), p(self.up), p(self.down),
                        p(self.shared_gate), p(self.shared_up), p(self.shared_down))


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not found at {LIB_PATH}; build it with "
                               "`python -m speculative_verify_router_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        D, W = ctypes.POINTER(_Desc), ctypes.POINTER(_Weights)
        KD, KB = ctypes.POINTER(_KvDesc), ctypes.POINTER(_KvBatch)
        sig = {
            "moe_version": (i32, []),
            "moe_strerror": (ctypes.c_char_p, [i32]),
            "moe_tensor_bytes": (i32, [i32, i64, i64, ctypes.POINTER(i64)]),
            "moe_workspace_bytes": (i32, [D, i32, ctypes.POINTER(sz)]),
            "moe_route": (i32, [D, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_layer_forward": (i32, [D, W, vp, i32, vp, vp, vp, vp, sz, vp]),
            "moe_layer_forward_timed": (i32, [D, W, vp, i32, vp, vp, vp, vp, sz, vp,
                                              ctypes.POINTER(vp), i32]),
            "moe_layer_forward_noalloc": (i32, [D, W, vp, i32, vp, vp, vp, vp]),
            "moe_stage_count": (i32, [D, i32]),
            "moe_stage_name": (ctypes.c_char_p, [D, i32, i32]),
            "moe_dequant_rows": (i32, [i32, vp, i64, i32, i64, i64, vp, vp]),
            "moe_accept_workspace_bytes": (i32, [i32, i64, ctypes.POINTER(sz)]),
            "moe_verify_accept": (i32, [vp, i32, i64, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "moe_kv_cache_bytes": (i32, [KD, i64, ctypes.POINTER(i64)]),
            "moe_kv_append": (i32, [KD, KB, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i32,
                                    vp, vp]),
            "moe_kv_attention_workspace_bytes": (i32, [KD, KB, ctypes.POINTER(sz)]),
            "moe_kv_attention": (i32, [KD, KB, i32, vp, i64, vp, i32, vp, vp, vp, sz, vp]),
            "moe_kv_read": (i32, [KD, KB, vp, i32, vp, vp, vp]),
            "moe_logprobs_workspace_bytes": (i32, [i32, i64, i32, ctypes.POINTER(sz)]),
            "moe_logprobs": (i32, [vp, i32, i32, i64, i64, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# Exported names of the C ABI (the header declares exactly these).
C_SYMBOLS = ("moe_version", "moe_strerror", "moe_tensor_bytes", "moe_workspace_bytes",
             "moe_route", "moe_layer_forward", "moe_layer_forward_timed",
             "moe_layer_forward_noalloc", "moe_stage_count",
             "moe_stage_name", "moe_dequant_rows", "moe_accept_workspace_bytes",
             "moe_verify_accept", "moe_kv_cache_bytes", "moe_kv_append",
             "moe_kv_attention_workspace_bytes", "moe_kv_attention", "moe_kv_read",
             "moe_logprobs_workspace_bytes", "moe_logprobs")


def _ptr(t: Optional[torch.Tensor], dtype) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != OK:
        raise MoeError(status, what)


def moe_version() -> int:
    return lib().moe_version()


def strerror(status: int) -> str:
    return lib().moe_strerror(status).decode()


def moe_strerror(status: int) -> str:
    return strerror(status)


def moe_tensor_bytes(dtype: str, rows: int, cols: int) -> int:
    out = ctypes.c_int64()
    _check(lib().moe_tensor_bytes(_DTYPES[dtype], rows, cols, ctypes.byref(out)), "moe_tensor_bytes")
    return out.value


def moe_workspace_bytes(desc: LayerDesc, max_tokens: int) -> int:
    out = ctypes.c_size_t()
    d = desc.c()
    _check(lib().moe_workspace_bytes(ctypes.byref(d), max_tokens, ctypes.byref(out)),
           "moe_workspace_bytes")
    return out.value


def moe_stage_count(desc: LayerDesc, n_tokens: int) -> int:
    d = desc.c()
    n = lib().moe_stage_count(ctypes.byref(d), n_tokens)
    if n <= 0:
        raise MoeError(-n, "moe_stage_count")
    return n


def moe_stage_name(desc: LayerDesc, n_tokens: int, i: int) -> Optional[str]:
    d = desc.c()
    s = lib().moe_stage_name(ctypes.byref(d), n_tokens, i)
    return None if s is None else s.decode()


# Leading workspace bytes that hold hand-off counters (zero between calls).
COUNTER_BYTES = 16384


def workspace(desc: LayerDesc, max_tokens: int, device="cuda") -> torch.Tensor:
    """A zero-filled device workspace of moe_workspace_bytes(desc, max_tokens)
    bytes (its counter page must start at zero; calls keep it so)."""
    n = max(moe_workspace_bytes(desc, max_tokens), COUNTER_BYTES)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_route(desc: LayerDesc, router: torch.Tensor, x: torch.Tensor, topk_ids: torch.Tensor,
              topk_w: torch.Tensor, expert_counts=None, expert_offsets=None, token_slots=None,
              active_experts=None, n_active=None, ws: torch.Tensor = None, stream=None):
    M = x.shape[0] if x.dim() == 2 else 0
    d = desc.c()
    if ws is None:
        ws = workspace(desc, M, x.device)
    i32 = torch.int32
    st = lib().moe_route(ctypes.byref(d), _ptr(router, torch.float32), _ptr(x, torch.float32), M,
                         _ptr(topk_ids, i32), _ptr(topk_w, torch.float32),
                         _ptr(expert_counts, i32), _ptr(expert_offsets, i32),
                         _ptr(token_slots, i32), _ptr(active_experts, i32), _ptr(n_active, i32),
                         _ptr(ws, torch.uint8), ws.numel(), _stream(stream))
    _check(st, "moe_route")


def moe_layer_forward(desc: LayerDesc, weights: LayerWeights, x: torch.Tensor, y: torch.Tensor,
                      topk_ids=None, topk_w=None, ws: torch.Tensor = None, stream=None):
    M = x.shape[0]
    d, w = desc.c(), weights.c()
    if ws is None:
        ws = workspace(desc, M, x.device)
    st = lib().moe_layer_forward(ctypes.byref(d), ctypes.byref(w), _ptr(x, torch.float32), M,
                                 _ptr(y, torch.float32), _ptr(topk_ids, torch.int32),
                                 _ptr(topk_w, torch.float32), _ptr(ws, torch.uint8), ws.numel(),
                                 _stream(stream))
    _check(st, "moe_layer_forward")


def moe_layer_forward_timed(desc: LayerDesc, weights: LayerWeights, x: torch.Tensor,
                            y: torch.Tensor, events: Sequence, topk_ids=None, topk_w=None,
                            ws: torch.Tensor = None, stream=None):
    """``events``: moe_stage_count(desc, M) + 1 raw hipEvent_t handles (ints)."""
    M = x.shape[0]
    d, w = desc.c(), weights.c()
    if ws is None:
        ws = workspace(desc, M, x.device)
    arr = (ctypes.c_void_p * len(events))(*events)
    st = lib().moe_layer_forward_timed(ctypes.byref(d), ctypes.byref(w), _ptr(x, torch.float32), M,
                                       _ptr(y, torch.float32), _ptr(topk_ids, torch.int32),
                                       _ptr(topk_w, torch.float32), _ptr(ws, torch.uint8),
                                       ws.numel(), _stream(stream), arr, len(events))
    _check(st, "moe_layer_forward_timed")


# Workspace bytes that moe_layer_forward_noalloc holds per GPU (MOE_NOALLOC_MAX_WORKSPACE).
NOALLOC_MAX_WORKSPACE = 8 << 20


def moe_layer_forward_noalloc(desc: LayerDesc, weights: LayerWeights, x: torch.Tensor,
                              y: torch.Tensor, topk_ids=None, topk_w=None, stream=None):
    """moe_layer_forward with the library's own per-GPU workspace (no allocation)."""
    M = x.shape[0]
    d, w = desc.c(), weights.c()
    st = lib().moe_layer_forward_noalloc(ctypes.byref(d), ctypes.byref(w), _ptr(x, torch.float32),
                                         M, _ptr(y, torch.float32), _ptr(topk_ids, torch.int32),
                                         _ptr(topk_w, torch.float32), _stream(stream))
    _check(st, "moe_layer_forward_noalloc")


class PreparedForward:
    """A moe_layer_forward call with its arguments marshalled once.

    The tensors are captured by reference (their device pointers are fixed);
    calling the object enqueues the layer again on the captured stream.
    ``events`` (raw hipEvent_t handles), if given per call, selects
    moe_layer_forward_timed.
    """

    def __init__(self, desc: LayerDesc, weights: LayerWeights, x: torch.Tensor, y: torch.Tensor,
                 topk_ids=None, topk_w=None, ws: torch.Tensor = None, stream=None):
        self._keep = (weights, x, y, topk_ids, topk_w)
        if ws is None:
            ws = workspace(desc, x.shape[0], x.device)
        self._ws = ws
        self._d = desc.c()
        self._w = weights.c()
        vp = ctypes.c_void_p
        self._args = (ctypes.byref(self._d), ctypes.byref(self._w), vp(_ptr(x, torch.float32)),
                      ctypes.c_int32(x.shape[0]), vp(_ptr(y, torch.float32)),
                      vp(_ptr(topk_ids, torch.int32)), vp(_ptr(topk_w, torch.float32)),
                      vp(_ptr(ws, torch.uint8)), ctypes.c_size_t(ws.numel()),
                      vp(_stream(stream)))
        self._f = lib().moe_layer_forward
        self._ft = lib().moe_layer_forward_timed

    def __call__(self, events=None):
        if events is None:
            st = self._f(*self._args)
        else:
            st = self._ft(*self._args, events, len(events))
        if st != OK:
            raise MoeError(st, "moe_layer_forward")


def moe_dequant_rows(dtype: str, tensor: torch.Tensor, rows: int, cols: int, row_start: int,
                     row_count: int, out: torch.Tensor, stream=None):
    st = lib().moe_dequant_rows(_DTYPES[dtype], _ptr(tensor, None), rows, cols, row_start,
                                row_count, _ptr(out, torch.float32), _stream(stream))
    _check(st, "moe_dequant_rows")


# include/moe_accept.h: greedy verify/accept of an MTP verify batch.
ACCEPT_MAX_ROWS = 64


def moe_accept_workspace_bytes(max_rows: int, vocab: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().moe_accept_workspace_bytes(max_rows, vocab, ctypes.byref(out)),
           "moe_accept_workspace_bytes")
    return out.value


def accept_workspace(max_rows: int, vocab: int, device="cuda") -> torch.Tensor:
    """A zero-filled device workspace for moe_verify_accept (its counter line
    must start at zero; calls keep it so)."""
    return torch.zeros(moe_accept_workspace_bytes(max_rows, vocab), dtype=torch.uint8,
                       device=device)


def moe_verify_accept(logits: torch.Tensor, drafts: Optional[torch.Tensor], tokens: torch.Tensor,
                      accepted: torch.Tensor, n_accepted: torch.Tensor,
                      verify_h: Optional[torch.Tensor] = None,
                      pending_h: Optional[torch.Tensor] = None, ws: torch.Tensor = None,
                      stream=None, n_rows: Optional[int] = None, vocab: Optional[int] = None):
    """logits [M][V] float32; drafts [M-1] int32 (None for M == 1); tokens,
    accepted [M] and n_accepted [1] int32 outputs; verify_h [M][h] and
    pending_h [h] float32, both or neither.  ``n_rows``/``vocab`` override
    the shape read from ``logits`` (for error-path tests)."""
    M = logits.shape[0] if n_rows is None else n_rows
    V = logits.shape[-1] if vocab is None else vocab
    if ws is None:
        ws = accept_workspace(max(M, 1), max(V, 1), logits.device)
    h_dim = 0 if verify_h is None else verify_h.shape[-1]
    i32 = torch.int32
    st = lib().moe_verify_accept(_ptr(logits, torch.float32), M, V, _ptr(drafts, i32),
                                 _ptr(verify_h, torch.float32), h_dim, _ptr(tokens, i32),
                                 _ptr(accepted, i32), _ptr(n_accepted, i32),
                                 _ptr(pending_h, torch.float32), _ptr(ws, torch.uint8), ws.numel(),
                                 _stream(stream))
    _check(st, "moe_verify_accept")


# include/moe_kv.h: paged 4-bit key/value cache, append and attention.
BF16, F16 = 6, 7
_ACT_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
KV_ROTARY_INTERLEAVED = 1
KV_COUNTER_BYTES = 16384


def _act_dtype(t: torch.Tensor) -> int:
    try:
        return _ACT_DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"expected float32, bfloat16 or float16, got {t.dtype}") from None


def _on(device: torch.device, t: Optional[torch.Tensor], dtype=None, shape=None,
        what: str = "tensor") -> Optional[int]:
    """The address of a contiguous tensor of `device` (None for None)."""
    if t is None:
        return None
    if t.device != device:
        raise ValueError(f"{what}: expected a tensor on {device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


def _rows(device: torch.device, t: torch.Tensor, dtype, shape, what: str):
    """Address and row stride of a [rows][heads][dim] tensor whose rows may lie apart."""
    if t.device != device:
        raise ValueError(f"{what}: expected a tensor on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    s, row = t.stride(), shape[1] * shape[2]
    if shape[0] == 0:
        return t.data_ptr(), row
    if s[2] != 1 or (s[1] != shape[2] and shape[1] != 1) or (s[0] < row and shape[0] != 1):
        raise ValueError(f"{what}: expected whole rows of heads, got strides {s}")
    return t.data_ptr(), (row if shape[0] == 1 else s[0])


def _current_stream_handle(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# torch's own lookup of the handle, without the Stream object around it (2 us of a 12 us call).
_current_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream_handle)


def _call_on(device: torch.device, stream, f, *args) -> int:
    """f(*args, stream) with `device` current; its current stream where none is given."""
    if device.type != "cuda":
        raise ValueError("expected a device tensor")
    index = device.index
    if stream is None:
        handle = _current_stream_handle(index)
    elif stream.device != device:
        raise ValueError(f"expected a stream of {device}, got one of {stream.device}")
    else:
        handle = stream.cuda_stream
    if index == torch.cuda.current_device():
        return f(*args, handle)
    with torch.cuda.device(device):
        return f(*args, handle)


def _check_bits(bits: int, **numbers):
    """ctypes would cut a larger number off in silence."""
    for name, n in numbers.items():
        if not -2 ** (bits - 1) <= n < 2 ** (bits - 1):
            raise ValueError(f"{name}: {n} does not fit {bits} bits")


def _check_int32(obj, *names):
    _check_bits(32, **{name: getattr(obj, name) for name in names})


def _default_workspace(stream, make, *args) -> torch.Tensor:
    """A workspace of the stream that will use it: filled there, and given back there."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


@dataclasses.dataclass(frozen=True)
class KvDesc:
    """Head layout and cache format of one attention layer (moe_kv_desc)."""
    n_heads: int
    n_kv_heads: int
    head_dim: int
    page_size: int = 64
    window: int = 0
    rotary_dims: int = 0
    rotary_interleaved: bool = False
    scale: float = 0.0  # 0: 1/sqrt(head_dim)
    norm_eps: float = 1e-6

    def __post_init__(self):
        _check_int32(self, "n_heads", "n_kv_heads", "head_dim", "page_size", "window", "rotary_dims")
        if self.scale != 0 and ctypes.c_float(self.scale).value == 0:
            raise ValueError(f"scale: {self.scale} is zero in 32 bits, which stands for 1/sqrt(head_dim)")
        # The fields never change, so the C struct is made once.
        object.__setattr__(self, "_c", _KvDesc(
            self.n_heads, self.n_kv_heads, self.head_dim, self.page_size, self.window,
            self.rotary_dims, KV_ROTARY_INTERLEAVED if self.rotary_interleaved else 0, self.scale,
            self.norm_eps))

    def c(self) -> _KvDesc:
        return self._c

    @property
    def page_bytes(self) -> int:
        """Bytes of one page of one key/value head."""
        return self.page_size * (self.head_dim + self.head_dim // 16)


@dataclasses.dataclass(frozen=True)
class KvBatch:
    """New rows of a batch of sequences (moe_kv_batch): int32 device tensors
    q_offsets [B+1], seq_lens [B] (new rows included), page_table [B][pages];
    max_rows: no sequence has more new rows.  The tensors are captured by
    reference, as PreparedForward does: write new lengths into them, or make
    another KvBatch."""
    q_offsets: torch.Tensor
    seq_lens: torch.Tensor
    page_table: torch.Tensor
    max_rows: int

    def __post_init__(self):
        i32, dev = torch.int32, self.page_table.device
        if self.page_table.dim() != 2:
            raise ValueError("page_table: expected [sequences][pages]")
        B, width = self.page_table.shape
        args = (width, _on(dev, self.q_offsets, i32, (B + 1,), "q_offsets"),
                _on(dev, self.seq_lens, i32, (B,), "seq_lens"),
                _on(dev, self.page_table, i32, None, "page_table"))
        _check_int32(self, "max_rows")
        object.__setattr__(self, "_args", args)
        object.__setattr__(self, "_device", dev)
        object.__setattr__(self, "_c", None)

    def c(self, n_tokens: int, device: Optional[torch.device] = None) -> _KvBatch:
        """The C struct for rows on `device` (None: sizes only)."""
        c = self._c
        if device is not None and device != self._device:
            raise ValueError(f"batch: expected tensors on {device}, got {self._device}")
        if c is None or c.n_tokens != n_tokens:
            c = _KvBatch(self.page_table.shape[0], n_tokens, self.max_rows, *self._args)
            object.__setattr__(self, "_c", c)
        return c


def moe_kv_cache_bytes(desc: KvDesc, n_pages: int) -> int:
    out = ctypes.c_int64()
    _check_bits(64, n_pages=n_pages)
    _check(lib().moe_kv_cache_bytes(desc.c(), n_pages, ctypes.byref(out)), "moe_kv_cache_bytes")
    return out.value


def kv_cache(desc: KvDesc, n_pages: int, device="cuda") -> torch.Tensor:
    """A cache of n_pages pages: uint8 [n_pages][n_kv_heads][page bytes], zeros."""
    moe_kv_cache_bytes(desc, n_pages)
    return torch.zeros((n_pages, desc.n_kv_heads, desc.page_bytes), dtype=torch.uint8, device=device)


def _cache(desc: KvDesc, cache: torch.Tensor, device: torch.device) -> int:
    return _on(device, cache, torch.uint8, (cache.shape[0], desc.n_kv_heads, desc.page_bytes), "cache")


def moe_kv_append(desc: KvDesc, batch: KvBatch, q: Optional[torch.Tensor], k: torch.Tensor,
                  v: torch.Tensor, cache: torch.Tensor, q_out: Optional[torch.Tensor],
                  q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
                  inv_freq: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None, stream=None):
    """q [T][heads][D] (or None, with q_out None), k and v [T][kv_heads][D] of one
    activation type, rows of q, k, v possibly apart (views of a fused projection);
    q_norm, k_norm [D], inv_freq [rotary/2] float32; positions [T] int32 (None: places)."""
    dev, dt, f32 = k.device, k.dtype, torch.float32
    T, D = k.shape[0], desc.head_dim
    kv = (T, desc.n_kv_heads, D)
    qp, qs, op = None, 0, None
    if q is not None:
        qp, qs = _rows(dev, q, dt, (T, desc.n_heads, D), "q")
    if q_out is not None:
        op = _on(dev, q_out, dt, (T, desc.n_heads, D), "q_out")
    kp, ks = _rows(dev, k, dt, kv, "k")
    vp, vs = _rows(dev, v, dt, kv, "v")
    st = _call_on(dev, stream, lib().moe_kv_append, desc.c(), batch.c(T, dev), _act_dtype(k), qp, qs, kp,
                  ks, vp, vs, _on(dev, q_norm, f32, (D,), "q_norm"),
                  _on(dev, k_norm, f32, (D,), "k_norm"),
                  _on(dev, inv_freq, f32, (desc.rotary_dims // 2,), "inv_freq"),
                  _on(dev, positions, torch.int32, (T,), "positions"), _cache(desc, cache, dev),
                  cache.shape[0], op)
    _check(st, "moe_kv_append")


def moe_kv_attention_workspace_bytes(desc: KvDesc, batch: KvBatch, n_tokens: int) -> int:
    out = ctypes.c_size_t()
    _check_bits(32, n_tokens=n_tokens)
    _check(lib().moe_kv_attention_workspace_bytes(desc.c(), batch.c(n_tokens), ctypes.byref(out)),
           "moe_kv_attention_workspace_bytes")
    return out.value


def kv_workspace(desc: KvDesc, batch: KvBatch, n_tokens: int) -> torch.Tensor:
    """A device workspace for moe_kv_attention on batches of up to this size (sequences, rows of one,
    table, n_tokens rows), its counters zeroed (calls keep them so)."""
    ws = torch.empty(moe_kv_attention_workspace_bytes(desc, batch, n_tokens), dtype=torch.uint8,
                     device=batch.page_table.device)
    ws[:KV_COUNTER_BYTES].zero_()
    return ws


def moe_kv_attention(desc: KvDesc, batch: KvBatch, q: torch.Tensor, cache: torch.Tensor,
                     out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None):
    """q and out [T][heads][D] of one activation type (rows of q possibly apart);
    lse [T][heads] float32."""
    dev = q.device
    T, shape = q.shape[0], (q.shape[0], desc.n_heads, desc.head_dim)
    if ws is None:
        ws = _default_workspace(stream, kv_workspace, desc, batch, T)
    qp, qs = _rows(dev, q, q.dtype, shape, "q")
    st = _call_on(dev, stream, lib().moe_kv_attention, desc.c(), batch.c(T, dev), _act_dtype(q), qp, qs,
                  _cache(desc, cache, dev), cache.shape[0], _on(dev, out, q.dtype, shape, "out"),
                  _on(dev, lse, torch.float32, shape[:2], "lse"),
                  _on(dev, ws, torch.uint8, None, "ws"), ws.numel())
    _check(st, "moe_kv_attention")


def moe_kv_read(desc: KvDesc, batch: KvBatch, cache: torch.Tensor, k_out: Optional[torch.Tensor],
                v_out: Optional[torch.Tensor], stream=None):
    """The stored rows of the batch as float32 [T][kv_heads][D] (either may be None)."""
    dev = cache.device
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("moe_kv_read: k_out or v_out is needed")
    shape = (some.shape[0], desc.n_kv_heads, desc.head_dim)
    st = _call_on(dev, stream, lib().moe_kv_read, desc.c(), batch.c(shape[0], dev),
                  _cache(desc, cache, dev), cache.shape[0],
                  _on(dev, k_out, torch.float32, shape, "k_out"),
                  _on(dev, v_out, torch.float32, shape, "v_out"))
    _check(st, "moe_kv_read")


# include/moe_logprobs.h: log probabilities, entropy and top alternatives.
LOGPROBS_MAX_TOP = 64


def moe_logprobs_workspace_bytes(max_rows: int, vocab: int, max_top: int = 0) -> int:
    out = ctypes.c_size_t()
    _check_bits(32, max_rows=max_rows, max_top=max_top)
    _check_bits(64, vocab=vocab)
    _check(lib().moe_logprobs_workspace_bytes(max_rows, vocab, max_top, ctypes.byref(out)),
           "moe_logprobs_workspace_bytes")
    return out.value


def logprobs_workspace(max_rows: int, vocab: int, max_top: int = 0, device="cuda") -> torch.Tensor:
    """A zero-filled device workspace for moe_logprobs (its counters must start
    at zero; calls keep them so)."""
    return torch.zeros(moe_logprobs_workspace_bytes(max_rows, vocab, max_top), dtype=torch.uint8,
                       device=device)


def moe_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor],
                 logprobs: Optional[torch.Tensor], entropy: Optional[torch.Tensor] = None,
                 top_ids: Optional[torch.Tensor] = None,
                 top_logprobs: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None):
    """logits [N][V] float32, bfloat16 or float16 (rows possibly apart); targets [N]
    int32 and logprobs [N] float32, both or neither; entropy [N] float32; top_ids
    int32 and top_logprobs float32 [N][k], k the number of alternatives."""
    dev, f32 = logits.device, torch.float32
    if logits.dim() != 2:
        raise ValueError(f"logits: expected [rows][vocabulary], got shape {tuple(logits.shape)}")
    N, V = logits.shape
    if N and V and logits.stride(1) != 1 and V != 1:
        raise ValueError(f"logits: expected whole rows, got strides {logits.stride()}")
    stride = logits.stride(0) if N > 1 else V
    some = top_ids if top_ids is not None else top_logprobs
    if some is not None and some.dim() != 2:
        raise ValueError("top_ids, top_logprobs: expected [rows][alternatives]")
    k = some.shape[1] if some is not None else 0
    if ws is None:
        ws = _default_workspace(stream, logprobs_workspace, N, V, k, dev)
    st = _call_on(dev, stream, lib().moe_logprobs, logits.data_ptr(), _act_dtype(logits), N, V,
                  stride, _on(dev, targets, torch.int32, (N,), "targets"),
                  _on(dev, logprobs, f32, (N,), "logprobs"),
                  _on(dev, entropy, f32, (N,), "entropy"), k,
                  _on(dev, top_ids, torch.int32, (N, k), "top_ids"),
                  _on(dev, top_logprobs, f32, (N, k), "top_logprobs"),
                  _on(dev, ws, torch.uint8, None, "ws"), ws.numel())
    _check(st, "moe_logprobs")
