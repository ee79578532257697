"""include/qmv/tuning.h without a GPU: every declared symbol is exported and
every precondition comes back as its status before anything is launched; the
Python layer refuses what does not fit."""
import ctypes
import math
import os
import re

import pytest
import torch

import quantized_matvec_amd as qmv
from quantized_matvec_amd import tuning as G
from quantized_matvec_amd.qmv import _Absmax

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -6
P = 0x7F0000010000
F32, F16, BF16 = 0, 1, 2
ref = ctypes.byref
BIG = 1 << 45


@pytest.fixture(scope="module")
def lib(qmvlib):
    return G.lib()


def weight(packed=P, absmax=P, rows=256, cols=512, bs=64, qt=0, dq=None):
    scales = _Absmax(absmax, None, None, None, None, 0) if dq is None else _Absmax(*dq)
    return G._Weight(packed, scales, rows, cols, bs, qt)


def lora(down=P, up=P, scale=P, count=3, rank=16):
    return G._Lora(down, up, scale, count, rank)


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "qmv", "tuning.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", text))
    assert names == {"qmv_lora_4bit_workspace", "qmv_lora_4bit", "qmv_lora_4bit_backward_workspace", "qmv_lora_4bit_backward",
                     "qmv_cross_entropy_4bit_workspace", "qmv_cross_entropy_4bit", "qmv_distill_4bit_workspace", "qmv_distill_4bit"}
    for n in names:
        assert hasattr(lib, n), n


WEIGHT_FAULTS = [(dict(packed=0), INVALID), (dict(absmax=0), INVALID), (dict(rows=0), INVALID), (dict(cols=0), INVALID),
                 (dict(rows=-1), INVALID), (dict(qt=2), INVALID), (dict(bs=48), UNSUPPORTED), (dict(bs=16), UNSUPPORTED),
                 (dict(bs=8192), UNSUPPORTED), (dict(cols=520), UNSUPPORTED), (dict(cols=544), UNSUPPORTED),
                 (dict(cols=1 << 22), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(packed=P + 8), ALIGN),
                 (dict(absmax=P + 4), ALIGN), (dict(dq=(P, P, P, P, P, 256)), INVALID), (dict(dq=(None, P, P, P, None, 256)), INVALID),
                 (dict(dq=(None, P, P, P, P, 100)), UNSUPPORTED), (dict(dq=(None, P + 1, P, P, P, 256)), ALIGN)]
LORA_FAULTS = [(dict(down=0), INVALID), (dict(up=0), INVALID), (dict(scale=0), INVALID), (dict(count=0), INVALID), (dict(rank=0), INVALID),
               (dict(rank=-8), INVALID), (dict(rank=12), UNSUPPORTED), (dict(rank=136), UNSUPPORTED), (dict(count=4097), UNSUPPORTED),
               (dict(down=P + 2), ALIGN), (dict(up=P + 8), ALIGN), (dict(scale=P + 2), ALIGN)]


def test_lora_preconditions(lib):
    def forward(w=None, l=None, x=P, dt=BF16, T=10, index=P, bias=None, y=P, ydt=BF16, ws=P, n=BIG):
        return lib.qmv_lora_4bit(x, dt, T, ref(w or weight()), ref(l or lora()), index, bias, y, ydt, ws, n, None)

    def backward(w=None, l=None, dy=P, x=P, dt=BF16, T=10, index=P, dx=P, dd=P, du=P, gdt=BF16, ws=P, n=BIG):
        return lib.qmv_lora_4bit_backward(dy, x, dt, T, ref(w or weight()), ref(l or lora()), index, dx, dd, du, gdt, ws, n, None)
    for change, want in WEIGHT_FAULTS:
        assert forward(w=weight(**change)) == want and backward(w=weight(**change)) == want, change
    for change, want in LORA_FAULTS:
        assert forward(l=lora(**change)) == want and backward(l=lora(**change)) == want, change
    for call in (forward, backward):
        assert call(T=0) == INVALID and call(T=-1) == INVALID and call(T=1 << 31) == UNSUPPORTED
        assert call(dt=F32) == UNSUPPORTED and call(dt=5) == INVALID and call(x=None) == INVALID and call(index=None) == INVALID
        assert call(index=P + 2) == ALIGN and call(x=P + 8) == ALIGN
        assert call(ws=None) == WORKSPACE and call(n=16) == WORKSPACE and call(ws=P + 8) == WORKSPACE
    assert forward(y=None) == INVALID and forward(y=P + 4) == ALIGN and forward(bias=P + 1) == ALIGN
    assert forward(ydt=F16) == UNSUPPORTED and forward(ydt=9) == INVALID
    for name in ("dy", "dx", "dd", "du"):
        assert backward(**{name: None}) == INVALID and backward(**{name: P + 8}) == ALIGN, name
    assert forward(w=weight(rows=1 << 22)) == UNSUPPORTED and backward(w=weight(rows=1 << 22)) == UNSUPPORTED
    assert backward(gdt=F16) == UNSUPPORTED and backward(w=weight(rows=257)) == UNSUPPORTED
    assert lib.qmv_lora_4bit(P, BF16, 10, None, ref(lora()), P, None, P, BF16, P, BIG, None) == INVALID
    assert lib.qmv_lora_4bit(P, BF16, 10, ref(weight()), None, P, None, P, BF16, P, BIG, None) == INVALID


def test_loss_preconditions(lib):
    def entropy(w=None, x=P, dt=BF16, T=10, target=P, dloss=None, loss=P, ldt=F32, dx=None, ws=P, n=BIG):
        return lib.qmv_cross_entropy_4bit(x, dt, T, ref(w or weight()), target, dloss, loss, ldt, dx, ws, n, None)

    def distill(w=None, x=P, dt=BF16, T=10, target=P, teacher=P, tdt=F32, k=4, tau=1.0, dloss=None, loss=P, ldt=F32, dx=None, ws=P, n=BIG):
        return lib.qmv_distill_4bit(x, dt, T, ref(w or weight()), target, teacher, tdt, k, tau, dloss, loss, ldt, dx, ws, n, None)
    for call in (entropy, distill):
        for change, want in WEIGHT_FAULTS:
            assert call(w=weight(**change)) == want, change
        assert call(T=0) == INVALID and call(T=1 << 31) == UNSUPPORTED and call(x=None) == INVALID and call(loss=None) == INVALID
        assert call(target=None) == INVALID and call(dloss=P) == INVALID and call(dx=P) == INVALID
        assert call(dt=F32) == UNSUPPORTED and call(ldt=F16) == UNSUPPORTED and call(ldt=4) == INVALID
        assert call(x=P + 8) == ALIGN and call(target=P + 4) == ALIGN and call(loss=P + 2) == ALIGN
        assert call(dx=P + 8, dloss=P) == ALIGN and call(dx=P, dloss=P + 2) == ALIGN
        assert call(ws=None) == WORKSPACE and call(n=16) == WORKSPACE and call(ws=P + 4) == WORKSPACE
    assert distill(teacher=None) == INVALID and distill(tdt=3) == INVALID and distill(k=0) == INVALID and distill(k=129) == UNSUPPORTED
    for tau in (0.0, -1.0, math.inf, math.nan, 1e-42):
        assert distill(tau=tau) == INVALID
    assert distill(teacher=P + 2) == ALIGN and distill(teacher=P + 1, tdt=BF16) == ALIGN


def test_workspaces(lib):
    for T in (1, 64, 65, 447, 448, 5000, 1 << 20):
        a = lib.qmv_lora_4bit_workspace(T, 14336, 4096, 64, 8, 16)
        b = lib.qmv_lora_4bit_backward_workspace(T, 14336, 4096, 64, 8, 16)
        c = lib.qmv_cross_entropy_4bit_workspace(T, 128256, 4096, 64, 0)
        d = lib.qmv_cross_entropy_4bit_workspace(T, 128256, 4096, 64, 1)
        assert 0 < a < 1 << 31 and 0 < b < 1 << 31 and 0 < c < d < 1 << 31, T
        assert lib.qmv_distill_4bit_workspace(T, 128256, 4096, 64, 128, 1) >= d
    assert lib.qmv_lora_4bit_workspace(0, 64, 64, 64, 1, 8) == 0 and lib.qmv_lora_4bit_workspace(4, 64, 64, 64, 1, 9) == 0
    assert lib.qmv_lora_4bit_backward_workspace(4, 65, 64, 64, 1, 8) == 0
    assert lib.qmv_cross_entropy_4bit_workspace(4, 65, 60, 32, 1) == 0 and lib.qmv_distill_4bit_workspace(4, 65, 64, 64, 129, 1) == 0


def test_python_layer_refuses():
    down, up = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 96, 8, dtype=torch.bfloat16)
    for d, u in ((down[0], up), (down, up[:1]), (down, up[..., :4]), (down.float(), up.float()), (down, up.half()),
                 (down[:0], up[:0]), (down[:, :4].contiguous(), up[..., :4].contiguous()), (down, up)):
        with pytest.raises(ValueError):  # the last: not on a GPU
            qmv.LoraAdapters(d, u)
    state = qmv.QuantState((96, 64), torch.bfloat16, 64, "nf4", absmax=torch.zeros(96))
    packed = torch.zeros(96 * 32, dtype=torch.uint8)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qmv.cross_entropy_4bit(x, packed, state, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        qmv.distill_4bit(x, packed, state, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))


def test_most_tokens_of_the_adapters_backward(lib):
    for T, want in (((1 << 22) - 1, WORKSPACE), (1 << 22, UNSUPPORTED)):
        assert lib.qmv_lora_4bit_backward(P, P, BF16, T, ref(weight()), ref(lora()), P, P, P, P, BF16, P, 16, None) == want
        assert (lib.qmv_lora_4bit_backward_workspace(T, 256, 128, 64, 3, 16) > 0) == (want == WORKSPACE)
