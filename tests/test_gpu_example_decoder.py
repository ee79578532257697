"""examples/decoder_4bit.py: what its calls leave behind and return, call by call.

The inputs and outputs of every append and attention call of a generation are
recorded.  All keys and values of a sequence, appended at once into a cache of
their own, must give the very bytes that the model's cache holds after its
prompt and its single steps; every attention output must lie within the bound
of kv_reference around the float64 attention over the cached values; and the
generation must repeat."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_reference as R
import quantized_matvec_amd as qmv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_4bit", os.path.join(ROOT, "examples", "decoder_4bit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype,name", [(torch.bfloat16, "bf16"), (torch.float16, "fp16")])
def test_generation(example, monkeypatch, dtype, name):
    g = torch.Generator().manual_seed(3)
    lengths, count = [50, 3, 17], 12
    prompts = [torch.randint(512, (n,), generator=g) for n in lengths]
    calls = []
    append, attend = qmv.kv_append_4bit, qmv.attention_4bit

    def record_append(cache, k, v, block_table, kv_len, cu_q=None, max_q=1, **kw):
        calls.append(dict(cache=cache, k=k.clone(), v=v.clone(), table=block_table, len=kv_len.tolist(),
                          cu=None if cu_q is None else cu_q.tolist()))
        return append(cache, k, v, block_table, kv_len, cu_q, max_q, **kw)

    def record_attend(q, cache, *a):
        out = attend(q, cache, *a)
        calls[-1].update(q=q.clone(), out=out.clone())
        return out
    monkeypatch.setattr(example.qmv, "kv_append_4bit", record_append)
    monkeypatch.setattr(example.qmv, "attention_4bit", record_attend)
    model = example.Decoder4bit(dtype=dtype)
    tokens, steps = example.generate(model, prompts, count)
    monkeypatch.undo()
    again, steps2 = example.generate(example.Decoder4bit(dtype=dtype), prompts, count)
    torch.cuda.synchronize()
    assert torch.equal(tokens, again) and torch.equal(steps, steps2)
    assert tokens.shape == (3, count) and torch.isfinite(steps.float()).all()

    hk, G, dim = model.kv_heads, model.heads // model.kv_heads, model.dim
    for cache in model.caches:
        mine = [c for c in calls if c["cache"] is cache]
        assert len(mine) == count
        for b, n in enumerate(lengths):
            total = n + count - 1
            rows = lambda c, x: c[x][c["cu"][b]:c["cu"][b + 1]] if c["cu"] else c[x][b:b + 1]
            k, v = (torch.cat([rows(c, x) for c in mine]) for x in "kv")
            assert k.shape[0] == total
            table = mine[0]["table"][b:b + 1]
            one = qmv.KVCache4bit(cache.num_pages, hk, cache.page_size, dim, cache.blocksize, "nf4", dtype)
            lens = torch.tensor([total], dtype=torch.int32, device="cuda")
            cu = torch.tensor([0, total], dtype=torch.int32, device="cuda")
            append(one, k, v, table, lens, cu, total, table=model.rope)
            held = [qmv.kv_dequantize_4bit(c, table, lens, total, cu_q=cu) for c in (one, cache)]
            torch.cuda.synchronize()
            assert torch.equal(held[0][0], held[1][0]) and torch.equal(held[0][1], held[1][1])
            # codes times scales in float64, from the cache's own bytes
            kd, vd = cached(cache, table[0].cpu().numpy(), total)
            for c in mine:
                q, out = rows(c, "q").double().cpu().numpy(), rows(c, "out").double().cpu().numpy()
                pos = c["len"][b] - q.shape[0] + np.arange(q.shape[0])
                for h in range(hk):
                    x = q[:, h * G:(h + 1) * G].reshape(-1, dim)
                    ref, bound = R.attend(x, kd[:, h], vd[:, h], dim ** -0.5, np.zeros(len(x), int), np.repeat(pos + 1, G))
                    bound = 1.01 * (bound + R.U_OUT[name] * np.abs(ref) + R.SUBNORMAL[name])
                    assert np.all(np.abs(out[:, h * G:(h + 1) * G].reshape(-1, dim) - ref) <= bound)


def cached(cache, pages, total):
    """Keys and values [total, heads, D] of a sequence in float64."""
    pages = pages[:-(-total // cache.page_size)]
    kc = cache.k_codes.cpu().numpy()[pages].transpose(0, 2, 1, 3)
    vc = cache.v_codes.cpu().numpy()[pages].transpose(0, 2, 4, 1, 3)
    out = []
    for codes, scales in ((kc, cache.k_scales), (vc, cache.v_scales)):
        codes = codes.reshape(-1, cache.heads, cache.head_dim // 2)[:total]
        s = scales.double().cpu().numpy()[pages].transpose(0, 3, 1, 2).reshape(-1, cache.heads, scales.shape[2])[:total]
        out.append(R.decode_rows(np.ascontiguousarray(codes), np.ascontiguousarray(s), cache.quant_type))
    return out
