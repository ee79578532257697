"""Arguments of the Python layer of the cache and of attention that are refused
by name, before any memory or kernel is asked for."""
import pytest

from quantized_matvec_amd import KVCache4bit


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
