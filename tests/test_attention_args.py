"""Arguments of the Python layer of the cache and of attention that are refused
by name, before any memory or kernel is asked for."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from quantized_matvec_amd import KVCache4bit, QmvError, attention


@pytest.mark.parametrize("head_dim,blocksize", [(128, 48), (128, 100), (96, 64), (160, 64), (128, 256), (64, 0), (64, -64), (65, 65),
                                                (0, 64), (-64, 32)])
def test_a_blocksize_that_does_not_divide_the_head(head_dim, blocksize):
    """Not the next size that does: the caller's blocks would be other ones."""
    with pytest.raises(ValueError, match="blocksize"):
        KVCache4bit(4, 2, 16, head_dim, blocksize)


@pytest.mark.parametrize("page_size", [0, -16, 8, 24, 100])
def test_a_page_size_without_whole_groups(page_size):
    with pytest.raises(ValueError, match="page_size"):
        KVCache4bit(4, 2, page_size, 64, 32)


def batch(max_q):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    return attention._batch(SimpleNamespace(device=torch.device("cpu")), i32(2, 4), i32(2), i32(3), max_q, 10)


@pytest.mark.parametrize("max_q", [2 ** 31, 2 ** 32 + 1, 2 ** 40, 2 ** 64 + 3])
def test_a_max_q_past_32_bits_bounds_nothing(qmvlib, max_q):
    """Not its low bits, which would leave tokens of a sequence unworked."""
    assert batch(max_q).max_q >= 10
    assert batch(None).max_q == 10 and batch(7).max_q == 7


@pytest.mark.parametrize("max_q", [0, -1, -2 ** 32 + 1])
def test_a_max_q_below_one(qmvlib, max_q):
    with pytest.raises(QmvError):
        batch(max_q)


# --------------------------------------------------------------------------
# Grids of 2^32 threads, which HIP does not launch.  Nothing is launched here
# either: on the small side there is no GPU, and the test does not run with one.
TOO_LARGE, LAUNCH, P = -7, -4, 0x7F0000010000
ref = ctypes.byref
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on addresses that are not there")


def heads(n, dim):
    return attention._Heads(P, n * dim, dim, n)


def sequences(count, max_q):
    return attention._Batch(P, 8192, P, P, count, 8192, max_q)


def status(call, max_q, count=1, kv=8, q=8, dim=128, rot=None, half=False):
    L, tokens = attention.lib(), max_q + count - 1
    c = attention._Cache(P, P, P, P, 10, kv, 16, dim, 32, 0, 2)
    b, hk, hq, rope = sequences(count, max_q), heads(kv, dim), heads(q, dim), attention._Rope(P, 100, rot or dim, 0)
    if call == "append":
        return L.qmv_kv_append_4bit(ref(c), ref(b), tokens, ref(hk), ref(hk), None, None, None, None)
    if call == "read":
        return L.qmv_kv_dequantize_4bit(ref(c), ref(b), tokens, ref(hk), ref(hk), None)
    if call == "attention":
        return L.qmv_attention_4bit(ref(hq), ref(c), ref(b), tokens, 0, 0.1, 1, 0, ref(hq), None, 0, None)
    return L.qmv_rotary(ref(hq), ref(hq), None, None, 2, tokens, dim, P, ref(rope), 0, None)


@no_gpu
@pytest.mark.parametrize("call,below,kw", [
    ("attention", 130816, dict(count=512, kv=32, q=32)),            # tiles of 256 rows, 512 threads each: 2^23 of them
    ("attention", (1 << 20) - 1, dict(kv=2, q=64, dim=160)),        # a wave a row: 2^26 rows
    ("rotary", (1 << 32) // (65 * 16) - 1, dict(q=64, rot=126)),    # 65 units of a head, four heads a thread
    ("append", 1 << 25, dict(kv=1)), ("read", 1 << 26, dict(kv=1))])
def test_grids_past_the_threads_of_a_launch(qmvlib, call, below, kw):
    assert status(call, below, **kw) == LAUNCH          # (no GPU)
    assert status(call, below * 8, **kw) == TOO_LARGE
    if call == "attention":
        step = 256 if kw.get("dim", 128) == 128 else 1
        assert status(call, below + step, **kw) == TOO_LARGE
