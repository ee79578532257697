"""Python binding of include/qmv/tuning.h (ctypes): low-rank adapters beside a
4-bit projection, and losses over a 4-bit vocabulary projection.

Argument marshalling only, as in ``qmv``: every step runs in the library's HIP
kernels on torch's current stream, and arguments that do not fit raise before
anything is launched.

    adapters = LoraAdapters(down, up, scale)         # [n, rank, K], [n, N, rank], [n]
    y = lora_4bit(x, packed, state, adapters, index)  # index [T]: each token's adapter, -1 for none
    dx, d_down, d_up = lora_4bit_backward(dy, x, packed, state, adapters, index)

    loss = cross_entropy_4bit(x, packed, state, target)               # [T]
    loss, dx = cross_entropy_4bit(x, packed, state, target, dloss)    # and the gradient of (dloss * loss).sum()
    loss, dx = distill_4bit(x, packed, state, ids, teacher, temperature, dloss)

The weights are frozen: gradients are those of activations and adapters.  A
call takes its workspace from torch's allocator for its own duration; results
repeat bit for bit.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Union

import torch

from .attention import _raw_stream
from .qmv import _DT, _QT, QuantState, _Absmax, _check, _check_state, _dev, lib as _lib

__all__ = ["LoraAdapters", "cross_entropy_4bit", "distill_4bit", "lora_4bit", "lora_4bit_backward"]

_vp, _i32, _i64, _sz, _int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int


class _Weight(ctypes.Structure):
    _fields_ = [("packed", _vp), ("scales", _Absmax), ("rows", _i64), ("cols", _i64), ("blocksize", _i32),
                ("quant_type", _int)]


class _Lora(ctypes.Structure):
    _fields_ = [("down", _vp), ("up", _vp), ("scale", _vp), ("count", _i32), ("rank", _i32)]


_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library with the signatures of tuning.h; raises if it has not
    been built."""
    global _LIB
    if _LIB is None:
        L = _lib()
        wp, lp = ctypes.POINTER(_Weight), ctypes.POINTER(_Lora)
        sig = {
            "qmv_lora_4bit_workspace": (_sz, [_i64, _i64, _i64, _i32, _i32, _i32]),
            "qmv_lora_4bit": (_int, [_vp, _int, _i64, wp, lp, _vp, _vp, _vp, _int, _vp, _sz, _vp]),
            "qmv_lora_4bit_backward_workspace": (_sz, [_i64, _i64, _i64, _i32, _i32, _i32]),
            "qmv_lora_4bit_backward": (_int, [_vp, _vp, _int, _i64, wp, lp, _vp, _vp, _vp, _vp, _int, _vp, _sz, _vp]),
            "qmv_cross_entropy_4bit_workspace": (_sz, [_i64, _i64, _i64, _i32, _i32]),
            "qmv_cross_entropy_4bit": (_int, [_vp, _int, _i64, wp, _vp, _vp, _vp, _int, _vp, _vp, _sz, _vp]),
            "qmv_distill_4bit_workspace": (_sz, [_i64, _i64, _i64, _i32, _i32, _i32]),
            "qmv_distill_4bit": (_int, [_vp, _int, _i64, wp, _vp, _vp, _int, _i32, ctypes.c_float, _vp, _vp, _int, _vp, _vp,
                                        _sz, _vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _LIB = L
    return _LIB


# --------------------------------------------------------------------------
# operands
# --------------------------------------------------------------------------
# A decode step is a handful of calls on small tensors, where the host decides:
# each attribute of a tensor is asked for once, and what fits is seen to fit
# before the checks that say what does not.
def _holds(t: torch.Tensor, n: int, dtype, device) -> bool:
    return t.numel() == n and t.dtype is dtype and t.device == device


def _weight(packed: torch.Tensor, state: QuantState, device):
    """The packed codes as the kernels take them, and the weight's descriptor."""
    shape = state.shape
    if len(shape) != 2:
        raise ValueError("the quantized weight must be 2-D [N, K]")
    rows, cols = shape
    n, bs = rows * cols, state.blocksize
    nb = -(-n // bs)
    dense = lambda t, n, dtype: _holds(t, n, dtype, device) and t.is_contiguous()
    q, a2, off, c2, bs2 = state.absmax_q, state.absmax2, state.offset, state.code2, state.blocksize2
    if state.absmax is not None:
        fits = q is None and a2 is None and off is None and c2 is None and dense(state.absmax, nb, torch.float32)
        scales = _Absmax(state.absmax.data_ptr(), None, None, None, None, 0) if fits else None
    else:
        fits = (q is not None and a2 is not None and off is not None and c2 is not None and dense(q, nb, torch.uint8)
                and dense(a2, -(-nb // bs2), torch.float32) and dense(off, 1, torch.float32) and dense(c2, 256, torch.float32))
        scales = _Absmax(None, q.data_ptr(), a2.data_ptr(), c2.data_ptr(), off.data_ptr(), bs2) if fits else None
    if not fits or not _holds(packed, (n + 1) // 2, torch.uint8, device):
        _check_state(packed, state, device)  # says what does not fit
        raise ValueError("the quantized weight's tensors do not fit its shape")
    packed = _dev(packed, "packed")
    return packed, _Weight(packed.data_ptr(), scales, rows, cols, bs, _QT[state.quant_type])


def _tokens(x: torch.Tensor, name: str, width: int) -> torch.Tensor:
    """Rows [T, width] of 16-bit values as the kernels take them (a copy of views that are not)."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dim() < 1 or x.shape[-1] != width:
        raise ValueError(f"{name} must have {width} elements in its last dimension, got {tuple(x.shape)}")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be bf16 or fp16, got {x.dtype}")
    return _dev(x, name).reshape(-1, width)


def _out(t: Optional[torch.Tensor], shape, dtype, device, name: str, align: int = 16) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    n = 1
    for s in shape:
        n *= s
    if t.dtype != dtype or t.device != device or t.numel() != n or not t.is_contiguous() or t.data_ptr() % align:
        raise ValueError(f"{name} must be a contiguous, {align}-byte aligned tensor of {n} values of {dtype} on {device}")
    return t


def _vector(t: torch.Tensor, n: int, dtype, device, name: str) -> torch.Tensor:
    """A contiguous tensor of n values of a type on the operands' device."""
    if t.dtype != dtype or t.numel() != n or t.device != device:
        raise ValueError(f"{name} must hold {n} values of {dtype} on {device}, got {t.numel()} of {t.dtype} on {t.device}")
    return t.contiguous()


def _call(name: str, device: torch.device, nbytes: int, call) -> None:
    """call(workspace, its size, stream) on the operands' device.  The workspace
    is the allocator's again afterwards, which hands it out to later work of
    this stream (of this graph, in a capture) only."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, device, nbytes, call)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    st = torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(index)
    _check(call(ws.data_ptr(), nbytes, st), name)


class LoraAdapters:
    """Adapters beside a projection [N, K], all of one rank (a multiple of 8 up
    to 128; smaller ones are padded with zeros): ``down`` [n, rank, K] and
    ``up`` [n, N, rank] in bf16 or fp16, ``scale`` a number or fp32 [n].  The
    tensors are kept, not copied: what an optimizer writes into them counts."""

    def __init__(self, down: torch.Tensor, up: torch.Tensor, scale: Union[float, torch.Tensor] = 1.0):
        if down.dim() != 3 or up.dim() != 3 or down.shape[0] != up.shape[0] or down.shape[1] != up.shape[2]:
            raise ValueError(f"down must be [n, rank, K] and up [n, N, rank], got {tuple(down.shape)} and {tuple(up.shape)}")
        if down.dtype not in (torch.bfloat16, torch.float16) or up.dtype != down.dtype:
            raise ValueError(f"down and up must both be bf16 or fp16, got {down.dtype} and {up.dtype}")
        n, rank, _ = down.shape
        if n == 0 or rank == 0 or rank % 8 or rank > 128:
            raise ValueError(f"at least one adapter, of a rank that is a multiple of 8 up to 128: got {n} of rank {rank}")
        if not isinstance(scale, torch.Tensor):
            scale = torch.full((n,), float(scale), dtype=torch.float32, device=down.device)
        if scale.shape != (n,) or scale.dtype != torch.float32:
            raise ValueError(f"scale must be a number or fp32 [{n}], got {scale.dtype} {tuple(scale.shape)}")
        for t in (down, up, scale):
            if not t.is_cuda or not t.is_contiguous() or t.device != down.device:
                raise ValueError("down, up and scale must be contiguous and on one GPU")
        if down.data_ptr() % 16 or up.data_ptr() % 16:
            raise ValueError("down and up must be 16-byte aligned")
        self.down, self.up, self.scale = down, up, scale
        self.count, self.rank, self.K, self.N = n, rank, down.shape[2], up.shape[1]
        self.dtype, self.device = down.dtype, down.device

    def _c(self) -> _Lora:
        return _Lora(self.down.data_ptr(), self.up.data_ptr(), self.scale.data_ptr(), self.count, self.rank)


def _lora_operands(x, name, width, packed, state, adapters, index):
    x2 = _tokens(x, name, width)
    packed, w = _weight(packed, state, x.device)
    if (adapters.N, adapters.K) != tuple(state.shape) or adapters.dtype != x.dtype or adapters.device != x.device:
        raise ValueError(f"the adapters are for a weight [{adapters.N}, {adapters.K}] and {adapters.dtype} on {adapters.device}")
    index = _vector(index, x2.shape[0], torch.int32, x.device, "index")
    return x2, packed, w, index


def lora_4bit(x: torch.Tensor, packed: torch.Tensor, state: QuantState, adapters: LoraAdapters, index: torch.Tensor,
              bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """y [T, N] = x [T, K] @ W_hat^T (+ bias [N]) + the token's adapter:
    ``index`` int32 [T] numbers them, and a token whose number is outside
    [0, n) has none.  One rounding, to x's type or fp32 (``out_dtype``)."""
    if len(state.shape) != 2:
        raise ValueError("the quantized weight must be 2-D [N, K]")
    N, K = state.shape
    x2, packed, w, index = _lora_operands(x, "x", K, packed, state, adapters, index)
    T = x2.shape[0]
    out_dtype = out.dtype if out is not None else (out_dtype or x.dtype)
    if out_dtype not in (x.dtype, torch.float32):
        raise ValueError(f"the output is of x's type or fp32, not {out_dtype}")
    out = _out(out, (T, N), out_dtype, x.device, "out")
    if bias is not None:
        bias = _vector(bias, N, x.dtype, x.device, "bias")
    if T == 0:
        return out
    L, l = lib(), adapters._c()
    need = L.qmv_lora_4bit_workspace(T, N, K, state.blocksize, adapters.count, adapters.rank)
    _call("lora_4bit", x.device, need, lambda ws, n, st: L.qmv_lora_4bit(
        x2.data_ptr(), _DT[x.dtype], T, ctypes.byref(w), ctypes.byref(l), index.data_ptr(),
        bias.data_ptr() if bias is not None else None, out.data_ptr(), _DT[out_dtype], ws, n, st))
    return out


def lora_4bit_backward(dy: torch.Tensor, x: torch.Tensor, packed: torch.Tensor, state: QuantState,
                       adapters: LoraAdapters, index: torch.Tensor, grad_dtype: Optional[torch.dtype] = None,
                       dx: Optional[torch.Tensor] = None, d_down: Optional[torch.Tensor] = None,
                       d_up: Optional[torch.Tensor] = None):
    """(dx [T, K], d_down [n, rank, K], d_up [n, N, rank]) from dy [T, N] and
    lora_4bit's x: the gradients of x and of the adapters, the latter in the
    adapters' type or fp32 (``grad_dtype``), zeros for adapters without tokens."""
    if len(state.shape) != 2:
        raise ValueError("the quantized weight must be 2-D [N, K]")
    N, K = state.shape
    dy2, packed, w, index = _lora_operands(dy, "dy", N, packed, state, adapters, index)
    x2 = _tokens(x, "x", K)
    T = dy2.shape[0]
    if x2.shape[0] != T or x.dtype != dy.dtype or x.device != dy.device:
        raise ValueError("x must have the tokens, type and device of dy")
    grad_dtype = d_down.dtype if d_down is not None else (grad_dtype or x.dtype)
    if grad_dtype not in (x.dtype, torch.float32):
        raise ValueError(f"the adapters' gradients are of their type or fp32, not {grad_dtype}")
    dx = _out(dx, (T, K), x.dtype, x.device, "dx")
    d_down = _out(d_down, adapters.down.shape, grad_dtype, x.device, "d_down")
    d_up = _out(d_up, adapters.up.shape, grad_dtype, x.device, "d_up")
    if T == 0:
        return dx, d_down.zero_(), d_up.zero_()
    L, l = lib(), adapters._c()
    need = L.qmv_lora_4bit_backward_workspace(T, N, K, state.blocksize, adapters.count, adapters.rank)
    _call("lora_4bit_backward", x.device, need, lambda ws, n, st: L.qmv_lora_4bit_backward(
        dy2.data_ptr(), x2.data_ptr(), _DT[x.dtype], T, ctypes.byref(w), ctypes.byref(l), index.data_ptr(), dx.data_ptr(),
        d_down.data_ptr(), d_up.data_ptr(), _DT[grad_dtype], ws, n, st))
    return dx, d_down, d_up


# --------------------------------------------------------------------------
# losses
# --------------------------------------------------------------------------
def _loss_operands(x, packed, state, dloss, loss_dtype, dx):
    if len(state.shape) != 2:
        raise ValueError("the quantized weight must be 2-D [V, K]")
    x2 = _tokens(x, "x", state.shape[1])
    packed, w = _weight(packed, state, x.device)
    T = x2.shape[0]
    loss_dtype = loss_dtype or x.dtype
    if loss_dtype not in (x.dtype, torch.float32):
        raise ValueError(f"the loss is of x's type or fp32, not {loss_dtype}")
    loss = torch.empty(T, dtype=loss_dtype, device=x.device)
    if dloss is not None:
        dloss = _vector(dloss, T, torch.float32, x.device, "dloss")
        dx = _out(dx, (T, state.shape[1]), x.dtype, x.device, "dx")
    elif dx is not None:
        raise ValueError("dx without dloss")
    return x2, packed, w, dloss, loss, dx


def _ptr(t):
    return None if t is None else t.data_ptr()


def cross_entropy_4bit(x: torch.Tensor, packed: torch.Tensor, state: QuantState, target: torch.Tensor,
                       dloss: Optional[torch.Tensor] = None, loss_dtype: Optional[torch.dtype] = None,
                       dx: Optional[torch.Tensor] = None):
    """Softmax cross entropy [T] of the logits x [T, K] @ W_hat^T [K, V] against
    ``target`` int64 [T]; a target outside [0, V) does not count (loss 0, zeros
    in dx).  With ``dloss`` fp32 [T], the gradient of each token's loss, the
    result is (loss, dx [T, K]).  The logits are never kept whole."""
    x2, packed, w, dloss, loss, dx = _loss_operands(x, packed, state, dloss, loss_dtype, dx)
    T = x2.shape[0]
    target = _vector(target, T, torch.int64, x.device, "target")
    if T:
        L = lib()
        need = L.qmv_cross_entropy_4bit_workspace(T, *state.shape, state.blocksize, dx is not None)
        _call("cross_entropy_4bit", x.device, need, lambda ws, n, st: L.qmv_cross_entropy_4bit(
            x2.data_ptr(), _DT[x.dtype], T, ctypes.byref(w), target.data_ptr(), _ptr(dloss), loss.data_ptr(),
            _DT[loss.dtype], _ptr(dx), ws, n, st))
    return loss if dx is None else (loss, dx)


def distill_4bit(x: torch.Tensor, packed: torch.Tensor, state: QuantState, ids: torch.Tensor, teacher: torch.Tensor,
                 temperature: float = 1.0, dloss: Optional[torch.Tensor] = None,
                 loss_dtype: Optional[torch.dtype] = None, dx: Optional[torch.Tensor] = None):
    """Divergence [T] of softmax(x @ W_hat^T / temperature) from the
    distribution softmax(teacher / temperature) over the ids of a teacher's
    largest logits: ``ids`` int64 [T, k] (an id outside [0, V) is no entry) and
    ``teacher`` [T, k], k up to 128.  The ids of a row differ: one that comes
    twice is two entries, each with its own log p in the loss.  ``dloss`` and the result as for
    cross_entropy_4bit."""
    x2, packed, w, dloss, loss, dx = _loss_operands(x, packed, state, dloss, loss_dtype, dx)
    T = x2.shape[0]
    if ids.dim() != 2 or ids.shape[0] != T or ids.shape[1] == 0 or teacher.shape != ids.shape or teacher.dtype not in _DT:
        raise ValueError(f"ids and teacher must be [{T}, k], teacher fp32, fp16 or bf16")
    k = ids.shape[1]
    ids = _vector(ids, T * k, torch.int64, x.device, "ids")
    teacher = _vector(teacher, T * k, teacher.dtype, x.device, "teacher")
    if T:
        L = lib()
        need = L.qmv_distill_4bit_workspace(T, *state.shape, state.blocksize, k, dx is not None)
        _call("distill_4bit", x.device, need, lambda ws, n, st: L.qmv_distill_4bit(
            x2.data_ptr(), _DT[x.dtype], T, ctypes.byref(w), ids.data_ptr(), teacher.data_ptr(), _DT[teacher.dtype], k,
            temperature, _ptr(dloss), loss.data_ptr(), _DT[loss.dtype], _ptr(dx), ws, n, st))
    return loss if dx is None else (loss, dx)
