"""What the calls of include/qmv/tuning.h may ask for in workspace, without a GPU."""
import pytest

from quantized_matvec_amd import tuning as G


@pytest.mark.parametrize("V,K", [(32000, 2048), (128256, 4096), (128256, 8192), (1 << 20, 8192), (1 << 20, 512), (1 << 22, 64)])
def test_losses_hold_no_more_than_2_26_logits(qmvlib, V, K):
    """A loss alone has little else: each token's and each 8192 columns' maximum and sum, and, from 448 tokens on,
    a piece of the decoded weight, 32768 rows at most.  Products that come in slices of the sum count for every slice."""
    L = G.lib()
    for T in (1, 16, 17, 33, 64, 65, 447, 448, 1792, 1793, 4096, 4097, 1 << 20):
        n = L.qmv_cross_entropy_4bit_workspace(T, V, K, 64, 0)
        decoded = 2 * 32768 * K if T >= 448 else 0
        assert 0 < n <= 4 * (1 << 26) + decoded + (1 << 20), (T, n)
