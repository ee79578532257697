"""Python binding of include/qmv/attention.h (ctypes): rotary positions, the
paged 4-bit key/value cache and attention over it.

Argument marshalling only, as in ``qmv``: every step runs in the library's HIP
kernels on torch's current stream, and arguments that do not fit raise before
anything is launched.

    freqs = rope_frequencies(128, theta=500000.0)
    table = rope_table(freqs, max_pos=8192, device="cuda")
    cache = KVCache4bit(num_pages=512, heads=8, page_size=64, head_dim=128, device="cuda")
    # each step: q, k, v of the new tokens (views of one projection are fine)
    q = kv_append_4bit(cache, k, v, block_table, kv_len, q=q, table=table)
    out = attention_4bit(q, cache, block_table, kv_len)

``block_table`` [batch, max_pages] int32 holds page numbers, ``kv_len``
[batch] int32 the tokens of each sequence in the cache, the new ones included.
With more than one new token for a sequence, ``cu_q`` [batch + 1] int32 holds
the offsets of each sequence's tokens among all new tokens and ``max_q`` the
most tokens of one sequence.  Rows of tokens that are past ``max_q``, or of no
sequence, are not written: new outputs hold anything there.

A batch that mixes prompts with single tokens is right in one call, but faster in
two: one kernel is chosen for all sequences, by ``max_q``.
"""
from __future__ import annotations

import ctypes
import operator
import threading
from typing import Optional

import torch

from .qmv import _DT, _QT, QmvError, _check, _stream as _stream_of, lib as _lib

__all__ = ["KVCache4bit", "attention_4bit", "kv_append_4bit", "kv_dequantize_4bit",
           "rope_frequencies", "rope_table", "rotary", "rotary_backward"]

_vp, _i32, _i64, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double
_SCALING = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32)]


class _Rope(ctypes.Structure):
    _fields_ = [("table", _vp), ("max_pos", _i64), ("rot_dim", _i32), ("interleaved", _i32)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("v_codes", _vp), ("k_scales", _vp), ("v_scales", _vp),
                ("num_pages", _i64), ("heads", _i32), ("page_size", _i32), ("head_dim", _i32),
                ("blocksize", _i32), ("quant_type", ctypes.c_int), ("dtype", ctypes.c_int)]


class _Batch(ctypes.Structure):
    _fields_ = [("block_table", _vp), ("table_stride", _i64), ("kv_len", _vp), ("cu_q", _vp),
                ("batch", _i32), ("max_pages", _i32), ("max_q", _i32)]


_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library with the signatures of attention.h; raises if it has
    not been built."""
    global _LIB
    if _LIB is None:
        L = _lib()
        hp, rp, cp, bp = map(ctypes.POINTER, (_Heads, _Rope, _Cache, _Batch))
        sig = {
            "qmv_rope_frequencies": (ctypes.c_int, [_i32, _f64, ctypes.c_int, _f64, _i64, _f64, _f64, _vp]),
            "qmv_rope_table": (ctypes.c_int, [_vp, _i32, _i64, _f64, _vp, _vp]),
            "qmv_rotary": (ctypes.c_int, [hp, hp, hp, hp, ctypes.c_int, _i64, _i32, _vp, rp, _i32, _vp]),
            "qmv_kv_append_4bit": (ctypes.c_int, [cp, bp, _i64, hp, hp, rp, hp, hp, _vp]),
            "qmv_kv_dequantize_4bit": (ctypes.c_int, [cp, bp, _i64, hp, hp, _vp]),
            "qmv_attention_4bit_workspace": (ctypes.c_size_t, [cp, bp, _i64, _i32, _i64, _i64]),
            "qmv_attention_4bit": (ctypes.c_int, [hp, cp, bp, _i64, _i64, ctypes.c_float, _i32, _i64, hp,
                                                  _vp, ctypes.c_size_t, _vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _LIB = L
    return _LIB


# --------------------------------------------------------------------------
# operands
#
# A decode step is a handful of calls on small tensors, where the host decides:
# each attribute of a tensor is asked for once, and a descriptor is made from it.
# --------------------------------------------------------------------------
_SIZE = {torch.float32: 4, torch.float16: 2, torch.bfloat16: 2}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_ref = ctypes.byref


def _stream(t: torch.Tensor) -> int:
    return _stream_of(t) if _raw_stream is None else _raw_stream(t.get_device())


def _rows(t: torch.Tensor, name: str, dtype=None):
    """A GPU tensor [tokens, heads, head_dim] as the kernels take it (unit
    stride in head_dim, the others multiples of 16 bytes; a copy where they are
    not), and its descriptor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(shape)}")
    dt = t.dtype
    if dtype is not None and dt != dtype:
        raise ValueError(f"{name} must be {dtype}, got {dt}")
    if dt not in _SIZE:
        raise ValueError(f"{name} must be fp32, fp16 or bf16, got {dt}")
    ts, hs, es = t.stride()
    p = t.data_ptr()
    if es != 1 or (((ts | hs) * _SIZE[dt]) | p) & 15:
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
        ts, hs, _ = t.stride()
        p = t.data_ptr()
    return t, _Heads(p, ts, hs, shape[1])


def _out(t: Optional[torch.Tensor], like: torch.Tensor, name: str):
    """The output tensor (a new one for None) and its descriptor."""
    shape = like.shape
    if t is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
        return t, _Heads(t.data_ptr(), shape[1] * shape[2], shape[2], shape[1])
    ts, hs, es = t.stride() if t.dim() == 3 else (0, 0, 0)
    p = t.data_ptr()
    if t.shape != shape or t.dtype != like.dtype or t.device != like.device or es != 1 or \
            (((ts | hs) * _SIZE[t.dtype]) | p) & 15 or (ts == 0 and shape[0] > 1) or (hs == 0 and shape[1] > 1):
        raise ValueError(f"{name} must have the shape, type and device of its input, unit stride in "
                         "head_dim and 16-byte aligned rows")
    return t, _Heads(p, ts, hs, shape[1])


def _rope(table: torch.Tensor, interleaved: bool, device) -> _Rope:
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2 or table.dtype != torch.float32 or \
            not table.is_contiguous() or table.device != device:
        raise ValueError("table must be a contiguous fp32 [max_pos, rot_dim / 2, 2] tensor on the "
                         "operands' device")
    return _Rope(table.data_ptr(), shape[0], 2 * shape[1], int(interleaved))


class KVCache4bit:
    """A paged cache of 4-bit keys and values (layout and sizes:
    include/qmv/attention.h).  ``blocksize`` divides ``head_dim``: heads of 96
    or 160 have blocks of 32.

    ``k_codes`` / ``v_codes`` uint8 and ``k_scales`` / ``v_scales`` in
    ``dtype``, the 16-bit type of the keys, values and queries."""

    def __init__(self, num_pages: int, heads: int, page_size: int, head_dim: int,
                 blocksize: int = 64, quant_type: str = "nf4",
                 dtype: torch.dtype = torch.bfloat16, device="cuda"):
        if head_dim <= 0 or head_dim % 2 or blocksize <= 0 or head_dim % blocksize:
            raise ValueError(f"blocksize must divide head_dim, an even number: got {blocksize} and {head_dim}")
        if page_size <= 0 or page_size % 16:
            raise ValueError(f"page_size must be a multiple of 16, got {page_size}")
        shape = (num_pages, heads, page_size, head_dim // 2)
        sshape = (num_pages, heads, head_dim // blocksize, page_size)
        kc = torch.zeros(shape, dtype=torch.uint8, device=device)
        vc = torch.zeros((num_pages, heads, page_size // 16, head_dim // 2, 16), dtype=torch.uint8,
                         device=device)
        self._set(kc, torch.zeros(sshape, dtype=dtype, device=device), vc,
                  torch.zeros(sshape, dtype=dtype, device=device), quant_type)

    @classmethod
    def from_tensors(cls, k_codes, k_scales, v_codes, v_scales, quant_type: str = "nf4"):
        """A cache over existing tensors (kept, not copied)."""
        self = cls.__new__(cls)
        self._set(k_codes, k_scales, v_codes, v_scales, quant_type)
        return self

    def _set(self, kc, ks, vc, vs, quant_type):
        if kc.dim() != 4 or ks.dim() != 4 or kc.dtype != torch.uint8 or vc.dtype != torch.uint8:
            raise ValueError("k_codes must be uint8 [pages, heads, page, D / 2], k_scales [pages, heads, blocks, page]")
        pages, heads, page, half = kc.shape
        if vc.shape != (pages, heads, page // 16, half, 16) or page % 16:
            raise ValueError(f"v_codes must be [pages, heads, page / 16, D / 2, 16], got {tuple(vc.shape)}")
        if ks.shape[:2] != (pages, heads) or ks.shape[3] != page or vs.shape != ks.shape or \
                ks.dtype != vs.dtype or ks.dtype not in _DT:
            raise ValueError("k_scales and v_scales must be [pages, heads, D / blocksize, page] of one type")
        if ks.shape[2] == 0 or (2 * half) % ks.shape[2]:
            raise ValueError("the blocks of a row must divide head_dim")
        for t in (kc, ks, vc, vs):
            if not t.is_cuda or not t.is_contiguous() or t.device != kc.device:
                raise ValueError("the cache's tensors must be contiguous and on one GPU")
        if quant_type not in _QT:
            raise ValueError(f"quant_type must be one of {sorted(_QT)}")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = kc, ks, vc, vs
        self.num_pages, self.heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.blocksize = self.head_dim // ks.shape[2]
        self.quant_type, self.dtype, self.device = quant_type, ks.dtype, kc.device
        self._c = _Cache(kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, heads, page,
                         self.head_dim, self.blocksize, _QT[quant_type], _DT[ks.dtype])

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))


def _size(value, name: str, least: int) -> int:
    """A count from the caller, cut off where the library's 32 bits end (no
    sequence is longer): ctypes would keep its low bits."""
    value = operator.index(value)
    if value < least:
        raise QmvError(-1, f"{name} must be at least {least}, got {value}")
    return min(value, 2 ** 31 - 1)


def _batch(cache: KVCache4bit, block_table, kv_len, cu_q, max_q, tokens: int) -> _Batch:
    dev = cache.device
    shape = block_table.shape
    if len(shape) != 2 or block_table.dtype != torch.int32 or block_table.device != dev:
        raise ValueError("block_table must be int32 [batch, max_pages] with unit stride, on the cache's device")
    n, pages = shape
    stride, unit = block_table.stride()
    if unit != 1 and pages > 1:
        raise ValueError("block_table must have unit stride along its pages")
    if kv_len.shape != (n,) or kv_len.dtype != torch.int32 or kv_len.device != dev or not kv_len.is_contiguous():
        raise ValueError(f"kv_len must be contiguous int32 [{n}] on the cache's device")
    cu = None
    if cu_q is None:
        if tokens != n:
            raise ValueError(f"without cu_q there is one token for each of the {n} sequences, got {tokens}")
        max_q = 1
    else:
        if cu_q.shape != (n + 1,) or cu_q.dtype != torch.int32 or cu_q.device != dev or not cu_q.is_contiguous():
            raise ValueError(f"cu_q must be contiguous int32 [{n + 1}] on the cache's device")
        cu = cu_q.data_ptr()
        max_q = tokens if max_q is None else _size(max_q, "max_q", 1)
    return _Batch(block_table.data_ptr(), stride, kv_len.data_ptr(), cu, n, pages, max_q)


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
def rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> list:
    """The rot_dim / 2 angles per position (float64).  ``scaling`` stretches
    them for contexts ``factor`` times as long: "linear" all alike, "base" by
    a larger base, "bands" only the pairs that turn less than ``beta_fast``
    times within ``original_len`` positions."""
    buf = (ctypes.c_double * max(rot_dim // 2, 1))()
    _check(lib().qmv_rope_frequencies(rot_dim, theta, _SCALING[scaling], factor, original_len, beta_fast,
                                      beta_slow, ctypes.cast(buf, _vp)), "rope_frequencies")
    return list(buf)


def rope_table(freqs, max_pos: int, gain: float = 1.0, device="cuda") -> torch.Tensor:
    """gain * (cos, sin) of every position below max_pos: fp32 [max_pos, rot_dim / 2, 2]."""
    freqs = [float(f) for f in freqs]
    table = torch.empty((max_pos, len(freqs), 2), dtype=torch.float32, device=device)
    if not table.is_cuda:
        raise ValueError("the table lives on a GPU")
    buf = (ctypes.c_double * max(len(freqs), 1))(*freqs)
    _check(lib().qmv_rope_table(ctypes.cast(buf, _vp), 2 * len(freqs), max_pos, gain, table.data_ptr(),
                                _stream(table)), "rope_table")
    return table


def _rotary(q, k, table, positions, interleaved, q_out, k_out, inverse, name):
    q, hq = _rows(q, "q")
    tokens, _, dim = q.shape
    dev = q.device
    q_out, hqo = _out(q_out, q, "q_out")
    hk = hko = None
    if k is not None:
        k, hk = _rows(k, "k", q.dtype)
        if k.shape[0] != tokens or k.shape[2] != dim or k.device != dev:
            raise ValueError("k must have the tokens, head_dim and device of q")
        k_out, hko = _out(k_out, k, "k_out")
        hk, hko = _ref(hk), _ref(hko)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if positions.shape != (tokens,) or positions.dtype != torch.int64 or positions.device != dev \
            or not positions.is_contiguous():
        raise ValueError(f"positions must be contiguous int64 [{tokens}] on the operands' device")
    rope = _rope(table, interleaved, dev)
    if tokens:
        _check(lib().qmv_rotary(_ref(hq), _ref(hqo), hk, hko, _DT[q.dtype], tokens, dim, positions.data_ptr(),
                                _ref(rope), inverse, _stream(q)), name)
    return q_out, k_out


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], table: torch.Tensor, positions: torch.Tensor,
           interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
           k_out: Optional[torch.Tensor] = None):
    """Queries and keys [tokens, heads, head_dim] turned by their positions
    (int64 [tokens]): (q_out, k_out).  The outputs may be the inputs; a
    position outside the table gives a row of zeros."""
    return _rotary(q, k, table, positions, interleaved, q_out, k_out, 0, "rotary")


def rotary_backward(dq: torch.Tensor, dk: Optional[torch.Tensor], table: torch.Tensor,
                    positions: torch.Tensor, interleaved: bool = False,
                    q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Gradients of rotary's inputs from those of its outputs."""
    return _rotary(dq, dk, table, positions, interleaved, q_out, k_out, 1, "rotary_backward")


# --------------------------------------------------------------------------
# the cache
# --------------------------------------------------------------------------
def kv_append_4bit(cache: KVCache4bit, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
                   kv_len: torch.Tensor, cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                   q: Optional[torch.Tensor] = None, table: Optional[torch.Tensor] = None,
                   interleaved: bool = False, q_out: Optional[torch.Tensor] = None):
    """Writes the new tokens' keys and values [tokens, heads, head_dim] into
    the cache, the keys turned by their positions when ``table`` is given.
    With ``q`` the queries are turned in the same launch and returned."""
    dev = cache.device
    k, hk = _rows(k, "k", cache.dtype)
    v, hv = _rows(v, "v", cache.dtype)
    tokens = k.shape[0]
    if k.shape[1:] != (cache.heads, cache.head_dim) or k.shape != v.shape or k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be [tokens, {cache.heads}, {cache.head_dim}] on the cache's device")
    kb = _batch(cache, block_table, kv_len, cu_q, max_q, tokens)
    rope = None if table is None else _ref(_rope(table, interleaved, dev))
    hq = hqo = None
    if q is not None:
        if table is None:
            raise ValueError("q is turned by the table: give both or neither")
        q, hq = _rows(q, "q", cache.dtype)
        if q.shape[0] != tokens or q.shape[2] != cache.head_dim or q.device != dev:
            raise ValueError("q must have the tokens, head_dim and device of k")
        q_out, hqo = _out(q_out, q, "q_out")
        hq, hqo = _ref(hq), _ref(hqo)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if tokens:
        _check(lib().qmv_kv_append_4bit(_ref(cache._c), _ref(kb), tokens, _ref(hk), _ref(hv), rope, hq, hqo,
                                        _stream(k)), "kv_append_4bit")
    return q_out


def kv_dequantize_4bit(cache: KVCache4bit, block_table: torch.Tensor, kv_len: torch.Tensor, tokens: int,
                       cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                       k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """The last tokens of each sequence (one each, or by ``cu_q``) as the
    cache holds them: (k, v), each [tokens, heads, head_dim]."""
    kb = _batch(cache, block_table, kv_len, cu_q, max_q, tokens)
    shape = (tokens, cache.heads, cache.head_dim)
    if k_out is None:
        k_out = cache.k_scales.new_empty(shape)
    elif k_out.shape != shape or k_out.dtype != cache.dtype or k_out.device != cache.device:
        raise ValueError("k_out must be [tokens, heads, head_dim] of the cache's type and device")
    k_out, hk = _out(k_out, k_out, "k_out")
    v_out, hv = _out(v_out, k_out, "v_out")
    if tokens:
        _check(lib().qmv_kv_dequantize_4bit(_ref(cache._c), _ref(kb), tokens, _ref(hk), _ref(hv), _stream(k_out)),
               "kv_dequantize_4bit")
    return k_out, v_out


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
_WS: dict = {}        # (device, stream) -> workspace
_WS_LOCKS: dict = {}


def _workspace(nbytes: int, device: torch.device, key) -> torch.Tensor:
    """The workspace of one stream; a larger request replaces it."""
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _WS[key] = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def _with_workspace(nbytes: int, device: torch.device, stream: int, enqueue) -> int:
    """enqueue(pointer of a workspace, or None).  Calls on a stream share its
    workspace and run in order there; a call is several kernels, so from the
    look at the workspace until they are all enqueued no other thread's call
    may enqueue any on this stream.  A call that is being captured gets a
    workspace of its own from the graph's memory, which lives as long as the
    graph does."""
    if nbytes == 0:
        return enqueue(None)
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return enqueue(ws.data_ptr())
    key = (device.index, stream)
    with _WS_LOCKS.get(key) or _WS_LOCKS.setdefault(key, threading.RLock()):
        return enqueue(_workspace(nbytes, device, key).data_ptr())


def attention_4bit(q: torch.Tensor, cache: KVCache4bit, block_table: torch.Tensor, kv_len: torch.Tensor,
                   cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None,
                   max_kv: Optional[int] = None, scale: Optional[float] = None, causal: bool = True,
                   window: int = 0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [tokens, q_heads, head_dim] = softmax(scale q K^T) V over the cached
    keys of each token's sequence (query head h reads cache head
    h / (q_heads / heads)).  ``scale`` defaults to head_dim ** -0.5, ``max_kv``
    is a host-side upper bound of kv_len, ``window`` > 0 keeps the last
    ``window`` keys of each token.  A token that sees no key gets zeros."""
    q, hq = _rows(q, "q", cache.dtype)
    tokens, heads, dim = q.shape
    if dim != cache.head_dim or heads == 0 or heads % cache.heads or q.device != cache.device:
        raise ValueError(f"q must be [tokens, a multiple of {cache.heads}, {cache.head_dim}] on the cache's device")
    out, ho = _out(out, q, "out")
    kb = _batch(cache, block_table, kv_len, cu_q, max_q, tokens)
    if tokens == 0:
        return out
    L = lib()
    cache_p, kb_p, st = _ref(cache._c), _ref(kb), _stream(q)
    max_kv = 0 if max_kv is None else max(_size(int(max_kv), "max_kv", 0), 1)
    window = _size(window, "window", 0)
    n = L.qmv_attention_4bit_workspace(cache_p, kb_p, tokens, heads, max_kv, window)
    scale = dim ** -0.5 if scale is None else scale
    _check(_with_workspace(n, q.device, st, lambda ws: L.qmv_attention_4bit(
        _ref(hq), cache_p, kb_p, tokens, max_kv, scale, int(causal), window, _ref(ho), ws, n, st)), "attention_4bit")
    return out
