"""attention_4bit with device-side lengths that no cache holds (nothing outside
the operands is read, and what the other sequences get is right) and with
host-side sizes that no integer of the library holds."""
import pytest
import torch

from quantized_matvec_amd import attention_4bit, qmv
from test_gpu_attention import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("dim", [64, 160])
@pytest.mark.parametrize("window", [1, 16, 300, 2 ** 31 - 1])
def test_lengths_past_the_table_with_a_window(new, dim, window):
    """The keys inside such a sequence's window begin near position 2^31, or
    anywhere between the table's end and there: none is in the cache."""
    cache, table, _, _ = make([100, 100], 2, dim, 32, 16, "bf16", "nf4", 61)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    q = torch.randn(2 * new, 4, dim, device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    call = lambda lens, **kw: attention_4bit(q, cache, table, lens, cu_q=cu, max_q=new, window=window, **kw)
    want = call(i32(100, 100))
    for length in (2 ** 31 - 1, 2 ** 31 - 40, 2 ** 31 - 1024, 2 ** 30, 1 << 16, 1 << 12):
        for kw in ({}, {"max_kv": 100}, {"max_kv": 2 ** 31 - 1}):
            out = call(i32(length, 100), **kw)
            torch.cuda.synchronize()
            # other lengths divide the work differently: fp16 weights (2^-11 of values of
            # up to 4 on both sides) and a rounding of the result
            assert torch.allclose(out[new:].float(), want[new:].float(), rtol=2.0 ** -7, atol=4e-3)
            if length - new - window > 112:      # 7 pages of 16: the window is past them
                assert (out[:new] == 0).all()


def test_windows_and_bounds_past_the_integers_are_unlimited():
    """A window or a bound of the lengths that passes 64 bits is a large one, not its low bits."""
    cache, table, _, _ = make([500, 100], 2, 64, 32, 16, "bf16", "nf4", 62)
    kl = torch.tensor([500, 100], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    q = torch.randn(5, 4, 64, device="cuda").to(torch.bfloat16)
    call = lambda **kw: attention_4bit(q, cache, table, kl, **{"cu_q": cu, "max_q": 3, **kw})
    want = call()
    for big in (2 ** 31, 2 ** 32 + 1, 2 ** 63, 2 ** 64 + 1, 2 ** 64 + 16):
        assert torch.allclose(call(window=big).float(), want.float(), rtol=2.0 ** -7, atol=4e-3)
        assert torch.equal(call(max_kv=big), want)
        assert torch.equal(call(max_q=big), want)
    for bad in (dict(max_kv=-1), dict(max_kv=-2 ** 64 + 100), dict(window=-1), dict(window=-2 ** 64 + 100)):
        with pytest.raises(qmv.QmvError):
            call(**bad)
    torch.cuda.synchronize()
