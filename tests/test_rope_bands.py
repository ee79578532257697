"""rope_frequencies(scaling="bands"): each pair against its own number of turns,
also where all pairs turn often, or none does."""
import math

import numpy as np
import pytest

from quantized_matvec_amd import rope_frequencies


@pytest.mark.parametrize("rot,theta", [(128, 10000.0), (64, 500000.0), (96, 10000.0), (16, 100.0)])
@pytest.mark.parametrize("original_len", [1, 64, 256, 4096, 32768, 131072, 1600000, 10 ** 9, 10 ** 12])
@pytest.mark.parametrize("factor,fast,slow", [(8.0, 32.0, 1.0), (16.0, 32.0, 1.0), (2.0, 4.0, 3.9), (40.0, 1e4, 1e-3)])
def test_each_pair_by_its_turns(qmvlib, rot, theta, original_len, factor, fast, slow):
    plain = np.array(rope_frequencies(rot, theta))
    got = np.array(rope_frequencies(rot, theta, "bands", factor, original_len, fast, slow))
    turns = original_len * plain / (2 * math.pi)
    # pair i turns turns[0] theta^(-2 i / rot) times: the index, a real number, that turns beta times
    index = lambda beta: 0.5 * rot * math.log(turns[0] / beta) / math.log(theta)
    first, last = math.floor(index(fast)), math.ceil(index(slow))
    i = np.arange(rot // 2)
    assert np.allclose(got[turns > fast * 1.0001], plain[turns > fast * 1.0001], rtol=1e-12)
    assert np.allclose(got[turns < slow * 0.9999], plain[turns < slow * 0.9999] / factor, rtol=1e-12)
    between = (i > first) & (i < last)
    slowed = (i - first) / max(last - first, 1e-3)
    want = plain * (1 - slowed) + plain / factor * slowed
    assert np.allclose(got[between], want[between], rtol=1e-9)
    assert np.all(got <= plain * (1 + 1e-12)) and np.all(got >= plain / factor * (1 - 1e-12))


def test_the_slowest_pair_is_not_divided_whole_while_it_turns(qmvlib):
    """131072 positions: pair 63 of 64 turns 2.41 times, between 1 and 32."""
    plain, got = np.array(rope_frequencies(128)), np.array(rope_frequencies(128, 10000.0, "bands", 8.0, original_len=131072))
    assert math.isclose(got[63] / plain[63], 0.37, rel_tol=1e-12)       # (63 - 45) of (70 - 45), 1 - 0.72 + 0.72 / 8
    assert math.isclose(got[58] / plain[58], 0.545, rel_tol=1e-12)
    assert np.array_equal(got[:46], plain[:46])
