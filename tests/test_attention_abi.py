"""include/qmv/attention.h without a GPU: every declared symbol is exported,
every precondition comes back as its status before anything is launched, the
rotary frequencies follow their formulas, and the one-comparison code search
of the cache append decides as the exact one does."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import oracle as O
from quantized_matvec_amd import attention as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN, LAUNCH, HIPERR, WORKSPACE, LARGE = 0, -1, -2, -3, -4, -5, -6, -7
P = 0x7F0000010000
F32, F16, BF16 = 0, 1, 2
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib(qmvlib):
    return A.lib()


def heads(n=8, ts=1024, hs=128, p=P):
    return A._Heads(p, ts, hs, n)


def rope(p=P, max_pos=100, rot=128, inter=0):
    return A._Rope(p, max_pos, rot, inter)


def cache(**k):
    d = dict(kc=P, vc=P, ks=P, vs=P, pages=10, heads=2, page=16, dim=128, bs=64, qt=0, dt=BF16)
    d.update(k)
    return A._Cache(*d.values())


def batch(**k):
    d = dict(bt=P, stride=4, kl=P, cu=None, batch=3, pages=4, max_q=1)
    d.update(k)
    return A._Batch(*d.values())


def test_exports_every_declared_symbol(lib):
    with open(os.path.join(ROOT, "include", "qmv", "attention.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", text))
    assert names == {"qmv_rope_frequencies", "qmv_rope_table", "qmv_rotary", "qmv_kv_append_4bit", "qmv_kv_dequantize_4bit",
                     "qmv_attention_4bit_workspace", "qmv_attention_4bit"}
    for n in names:
        assert hasattr(lib, n), n


def test_rotary_preconditions(lib):
    def call(q=None, qo=None, k=None, ko=None, dt=BF16, tokens=10, dim=128, pos=P, r=None):
        p = lambda x: None if x is None else ref(x)
        return lib.qmv_rotary(ref(q or heads()), ref(qo or heads()), p(k), p(ko), dt, tokens, dim, pos, ref(r or rope()), 0, None)
    assert call(tokens=0) == INVALID and call(tokens=1 << 31) == INVALID
    assert call(dt=7) == INVALID and call(pos=None) == INVALID
    assert call(k=heads()) == INVALID and call(ko=heads()) == INVALID
    assert call(dim=100) == UNSUPPORTED and call(dim=8192) == UNSUPPORTED
    assert call(q=heads(p=0)) == INVALID and call(q=heads(n=0)) == INVALID and call(q=heads(n=4)) == INVALID
    assert call(q=heads(p=P + 8)) == ALIGN and call(q=heads(ts=1028)) == ALIGN and call(qo=heads(hs=132)) == ALIGN
    assert call(q=heads(ts=-1024)) == INVALID and call(pos=P + 4) == ALIGN
    assert call(r=rope(rot=3)) == INVALID and call(r=rope(rot=130)) == INVALID and call(r=rope(max_pos=0)) == INVALID
    assert call(r=rope(p=0)) == INVALID and call(r=rope(p=P + 8)) == ALIGN
    assert call(tokens=(1 << 31) - 1, q=heads(n=60000), qo=heads(n=60000)) == LARGE
    assert lib.qmv_rotary(None, ref(heads()), None, None, BF16, 10, 128, P, ref(rope()), 0, None) == INVALID
    assert lib.qmv_rotary(ref(heads()), ref(heads()), None, None, BF16, 10, 128, P, None, 0, None) == INVALID


CACHE_FAULTS = [(dict(pages=0), INVALID), (dict(heads=0), INVALID), (dict(qt=3), INVALID), (dict(dt=9), INVALID),
                (dict(dt=F32), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
                (dict(dim=48), UNSUPPORTED), (dict(dim=288), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(bs=16), UNSUPPORTED),
                (dict(bs=48), UNSUPPORTED), (dict(bs=256), UNSUPPORTED), (dict(dim=96, bs=64), UNSUPPORTED), (dict(kc=0), INVALID),
                (dict(vs=0), INVALID), (dict(vc=P + 4), ALIGN), (dict(ks=P + 2), ALIGN), (dict(pages=1 << 40), INVALID)]
BATCH_FAULTS = [(dict(bt=0), INVALID), (dict(kl=0), INVALID), (dict(batch=0), INVALID), (dict(pages=0), INVALID),
                (dict(max_q=0), INVALID), (dict(stride=3), INVALID), (dict(bt=P + 2), ALIGN), (dict(cu=P + 2), ALIGN),
                (dict(batch=4), INVALID), (dict(batch=65536, cu=P), UNSUPPORTED)]


def test_append_and_dequantize_preconditions(lib):
    def append(c=None, b=None, k=None, v=None, r=None, q=None, qo=None, tokens=3):
        p = lambda x: None if x is None else ref(x)
        return lib.qmv_kv_append_4bit(ref(c or cache()), ref(b or batch()), tokens, ref(k or heads(2)), ref(v or heads(2)), p(r),
                                      p(q), p(qo), None)

    def read(c=None, b=None, k=None, v=None, tokens=3):
        return lib.qmv_kv_dequantize_4bit(ref(c or cache()), ref(b or batch()), tokens, ref(k or heads(2)), ref(v or heads(2)), None)
    for change, want in CACHE_FAULTS:
        assert append(c=cache(**change)) == want and read(c=cache(**change)) == want, change
    for change, want in BATCH_FAULTS:
        assert append(b=batch(**change)) == want and read(b=batch(**change)) == want, change
    for call in (append, read):
        assert call(tokens=0) == INVALID and call(tokens=1 << 31) == INVALID and call(tokens=2) == INVALID
        assert call(k=heads(3)) == INVALID and call(v=heads(1)) == INVALID and call(v=heads(2, p=P + 4)) == ALIGN
        assert call(k=heads(2, ts=1027)) == ALIGN
    assert append(q=heads(), r=rope()) == INVALID and append(q=heads(), qo=heads()) == INVALID
    assert append(q=heads(), qo=heads(4), r=rope()) == INVALID
    assert append(r=rope(rot=130)) == INVALID and append(r=rope(rot=0)) == INVALID


def test_attention_preconditions(lib):
    def call(q=None, c=None, b=None, tokens=3, max_kv=0, scale=0.1, causal=1, window=0, out=None, ws=P, wsb=1 << 40):
        return lib.qmv_attention_4bit(ref(q or heads()), ref(c or cache()), ref(b or batch()), tokens, max_kv, scale, causal, window,
                                      ref(out or heads()), ws, wsb, None)
    for change, want in CACHE_FAULTS:
        assert call(c=cache(**change)) == want, change
    for change, want in BATCH_FAULTS:
        assert call(b=batch(**change)) == want, change
    assert call(tokens=0) == INVALID and call(tokens=4) == INVALID
    assert call(q=heads(7), out=heads(7)) == INVALID and call(q=heads(4)) == INVALID
    assert call(out=heads(p=P + 2)) == ALIGN and call(q=heads(ts=1025)) == ALIGN
    assert call(max_kv=-1) == INVALID and call(window=-1) == INVALID and call(window=4, causal=0) == INVALID
    for s in (math.nan, math.inf, -math.inf):
        assert call(scale=s) == INVALID


def test_attention_workspace(lib):
    """The size is a bound that the call checks, and 0 for arguments it refuses."""
    long = dict(pages=4096, stride=4096, batch=1)
    n = lib.qmv_attention_4bit_workspace(ref(cache()), ref(batch(**long)), 1, 8, 0, 0)
    b = batch(**long)
    args = lambda ws, wsb: lib.qmv_attention_4bit(ref(heads()), ref(cache()), ref(b), 1, 0, 0.1, 1, 0, ref(heads()), ws, wsb, None)
    if n:
        assert args(P, n - 1) == WORKSPACE and args(None, n) == WORKSPACE and args(P + 4, n) == ALIGN
    f = lib.qmv_attention_4bit_workspace
    for bad in ((cache(dim=48), batch(), 3, 8, 0, 0), (cache(), batch(batch=0), 3, 8, 0, 0), (cache(), batch(), 3, 7, 0, 0),
                (cache(), batch(), 3, 0, 0, 0), (cache(), batch(), 3, 8, -1, 0), (cache(), batch(), 3, 8, 0, -1)):
        assert f(ref(bad[0]), ref(bad[1]), *bad[2:]) == 0


def test_rope_frequencies():
    assert A.rope_frequencies(8) == [10000.0 ** (-2.0 * i / 8) for i in range(4)]
    plain = np.array(A.rope_frequencies(128, 500000.0))
    assert np.allclose(plain, 500000.0 ** (-np.arange(64) / 64.0), rtol=1e-15)
    assert np.allclose(A.rope_frequencies(128, 500000.0, "linear", 8.0), plain / 8, rtol=1e-15)
    base = np.array(A.rope_frequencies(128, 500000.0, "base", 8.0))
    assert base[0] == 1.0 and math.isclose(base[-1], plain[-1] / 8, rel_tol=1e-12)     # the slowest pair stretches by factor
    assert np.all(np.diff(np.log(base / plain)) < 0)
    bands = np.array(A.rope_frequencies(128, 10000.0, "bands", 16.0, original_len=4096, beta_fast=32, beta_slow=1))
    p = np.array(A.rope_frequencies(128, 10000.0))
    turns = 4096 * p / (2 * math.pi)
    assert np.allclose(bands[turns > 40], p[turns > 40]) and np.allclose(bands[turns < 0.8], p[turns < 0.8] / 16)
    mid = (turns < 30) & (turns > 1.2)
    share = (bands[mid] - p[mid] / 16) / (p[mid] - p[mid] / 16)                        # falls evenly in the pair's index
    assert np.all(share > 0) and np.all(share < 1) and np.allclose(np.diff(share), np.diff(share)[0])
    assert np.allclose(A.rope_frequencies(128, 10000.0, "bands", 1.0, original_len=4096), p)


def test_rope_frequencies_preconditions(lib):
    buf = ctypes.cast((ctypes.c_double * 64)(), ctypes.c_void_p)
    f = lambda *a: lib.qmv_rope_frequencies(*a, buf)
    assert f(128, 1e4, 0, 0.0, 0, 0.0, 0.0) == OK
    for bad in ((0, 1e4, 0, 1.0, 0, 1.0, 0.5), (7, 1e4, 0, 1.0, 0, 1.0, 0.5), (8, 0.0, 0, 1.0, 0, 1.0, 0.5),
                (8, math.nan, 0, 1.0, 0, 1.0, 0.5), (8, 1e4, 4, 1.0, 0, 1.0, 0.5), (8, 1e4, 1, 0.5, 0, 1.0, 0.5),
                (8, 1e4, 1, math.inf, 0, 1.0, 0.5), (2, 1e4, 2, 2.0, 0, 1.0, 0.5), (8, 1e4, 3, 2.0, 0, 32.0, 1.0),
                (8, 1e4, 3, 2.0, 4096, 1.0, 1.0), (8, 1e4, 3, 2.0, 4096, 32.0, 0.0), (8, 1.0, 3, 2.0, 4096, 32.0, 1.0)):
        assert f(*bad) == INVALID, bad
    assert lib.qmv_rope_frequencies(8, 1e4, 0, 1.0, 0, 1.0, 0.5, None) == INVALID
    t = lambda rot, n, gain, p: lib.qmv_rope_table(buf, rot, n, gain, p, None)
    assert t(3, 10, 1.0, P) == INVALID and t(128, 0, 1.0, P) == INVALID and t(128, 10, math.nan, P) == INVALID
    assert t(258, 10, 1.0, P) == UNSUPPORTED and t(128, 10, 1.0, P + 8) == ALIGN and t(128, 10, 1.0, None) == INVALID


@pytest.mark.parametrize("qt", ["nf4", "fp4"])
@pytest.mark.parametrize("bits", [8, 11])
def test_one_fp32_comparison_decides_exactly(qt, bits):
    """For every significand of a block maximum a and every midpoint m: each x
    of as many bits around a m compares with fp32(a fp32(m)) as with a m."""
    t = np.unique(O.code_table(qt).astype(np.float64))
    mids = (t[1:] + t[:-1]) / 2
    a = np.arange(1 << (bits - 1), 1 << bits).astype(np.float64)
    for m in mids:
        exact = a * m                                            # 11 + 25 bits: exact in float64
        fast = (a.astype(np.float32) * np.float32(m)).astype(np.float64)
        ulp = 2.0 ** (np.floor(np.log2(np.abs(exact))) - bits + 1)
        for d in (-2, -1, 0, 1, 2):
            x = (np.floor(exact / ulp) + d) * ulp
            above = (x > exact, x > fast) if m > 0 else (x >= exact, x >= fast)
            assert np.array_equal(*above), (m, d)
