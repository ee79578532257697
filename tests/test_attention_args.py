"""Arguments of the Python layer of the cache and of attention that are refused
by name, before any memory or kernel is asked for."""
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
