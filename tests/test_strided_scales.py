"""Scales with strides of their own (every other value of a tensor, one value
expanded) are refused before anything is launched: the kernels read them as contiguous."""
import pytest
import torch

import quantized_matvec_amd as qmv
from quantized_matvec_amd import qmv as Q
from quantized_matvec_amd import tuning as G

N, K, BS = 96, 64, 64
NB = N * K // BS


def state(device, **change):
    parts = dict(absmax_q=torch.zeros(NB, dtype=torch.uint8), absmax2=torch.ones(2), offset=torch.ones(1), code2=torch.ones(256))
    parts["absmax2"] = torch.ones(-(-NB // 64))
    plain = "absmax" in change
    parts = {"absmax": None} if plain else parts
    parts.update(change)
    parts = {k: v.to(device) if v.is_contiguous() else torch.as_strided(torch.ones(4096, device=device).to(v.dtype), v.shape, v.stride())
             for k, v in parts.items()}
    return qmv.QuantState((N, K), torch.bfloat16, BS, "nf4", blocksize2=64, **parts)


STRIDED = {"absmax, every other": dict(absmax=torch.ones(2 * NB)[::2]), "absmax, expanded": dict(absmax=torch.ones(1).expand(NB)),
           "absmax, transposed": dict(absmax=torch.ones(8, NB // 8).t()),
           "absmax_q, every other": dict(absmax_q=torch.zeros(2 * NB, dtype=torch.uint8)[::2]),
           "absmax2, expanded": dict(absmax2=torch.ones(1).expand(-(-NB // 64))), "code2, every other": dict(code2=torch.ones(512)[::2])}


@pytest.mark.parametrize("kind", sorted(STRIDED))
def test_refused(kind):
    s = state("cpu", **STRIDED[kind])
    packed = torch.zeros(N * K // 2, dtype=torch.uint8)
    for check in (lambda: Q._check_state(packed, s, packed.device), lambda: G._weight(packed, s, packed.device),
                  lambda: qmv.dequantize_absmax(s)):
        with pytest.raises(ValueError, match="contiguous"):
            check()
    for fine in (state("cpu"), state("cpu", absmax=torch.ones(NB)), state("cpu", absmax=torch.ones(8, NB // 8))):
        Q._check_state(packed, fine, packed.device)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", sorted(STRIDED))
def test_refused_by_every_call(kind):
    s = state("cuda", **STRIDED[kind])
    packed = torch.zeros(N * K // 2, dtype=torch.uint8, device="cuda")
    x, dy = torch.zeros(4, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, N, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    index = ids.int()
    a = qmv.LoraAdapters(torch.zeros(1, 8, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, N, 8, dtype=torch.bfloat16, device="cuda"))
    for call in (lambda: qmv.gemv_4bit(x, packed, s), lambda: qmv.gemm_4bit(x, packed, s), lambda: Q.gemm_4bit_backward(dy, packed, s),
                 lambda: qmv.dequantize_4bit(packed, s), lambda: qmv.dequantize_absmax(s), lambda: Q.embedding_4bit(ids, packed, s), lambda: qmv.lora_4bit(x, packed, s, a, index),
                 lambda: qmv.lora_4bit_backward(dy, x, packed, s, a, index), lambda: qmv.cross_entropy_4bit(x, packed, s, ids),
                 lambda: qmv.distill_4bit(x, packed, s, ids[:, None], ids[:, None].float())):
        with pytest.raises(ValueError, match="contiguous"):
            call()


@pytest.mark.gpu
def test_strided_codes_are_copied():
    """The packed codes may have strides: a call copies them."""
    s = state("cuda", absmax=torch.ones(NB))
    g = torch.Generator(device="cuda").manual_seed(1)
    packed = torch.randint(256, (N * K // 2, 2), generator=g, device="cuda", dtype=torch.uint8)
    x, ids = torch.randn(4, K, generator=g, device="cuda").bfloat16(), torch.arange(4, device="cuda")
    for call in (qmv.gemm_4bit, lambda *a: qmv.cross_entropy_4bit(*a, ids)):
        assert torch.equal(call(x, packed[:, 1], s), call(x, packed[:, 1].contiguous(), s))
