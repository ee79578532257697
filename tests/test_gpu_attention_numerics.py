"""attention_4bit on inputs that its reduced formats could get wrong: sums over
many keys that cancel, second terms of fp16 operands, keys and values of very
different size side by side, infinities and NaN in keys and values that a row
does not see, very large scores.

Relative norms here are over all outputs of a call.  With u the measured error
of rounding the exact result to the output's type, a kernel whose own error has
the relative norm e is at sqrt(u^2 + e^2): the two are independent."""
import numpy as np
import pytest
import torch

import kv_reference as R
from quantized_matvec_amd import KVCache4bit, attention_4bit, kv_append_4bit
from test_gpu_attention import TDT, check, make

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(L, hk, dim, bs, dt, qt, seed, k_gain=1.0, v_gain=1.0, page=64):
    """One sequence of L normal rows, appended, and its cached rows in float64 [L, hk, D]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = lambda gain: (torch.randn(L, hk, dim, generator=g, device="cuda") * gain).to(TDT[dt])
    pages = -(-L // page)
    cache = KVCache4bit(pages, hk, page, dim, bs, qt, TDT[dt])
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    kv_append_4bit(cache, rows(k_gain), rows(v_gain), table, i32([L]), cu_q=i32([0, L]))
    return cache, table, *cached(cache, table, L)


def cached(cache, table, L):
    pages = table[0].cpu().numpy()
    kc = cache.k_codes.cpu().numpy()[pages].transpose(0, 2, 1, 3)
    vc = cache.v_codes.cpu().numpy()[pages].transpose(0, 2, 4, 1, 3)
    out = []
    for codes, scales in ((kc, cache.k_scales), (vc, cache.v_scales)):
        codes = codes.reshape(-1, cache.heads, cache.head_dim // 2)[:L]
        s = scales.double().cpu().numpy()[pages].transpose(0, 3, 1, 2).reshape(-1, cache.heads, scales.shape[2])[:L]
        out.append(R.decode_rows(np.ascontiguousarray(codes), np.ascontiguousarray(s), cache.quant_type))
    return out


def norms(got, want, dt):
    """Relative norms of got's error and of rounding want to the type."""
    rounded = torch.from_numpy(want).to(TDT[dt]).double().numpy()
    size = np.linalg.norm(want)
    return np.linalg.norm(got.double().cpu().numpy() - want) / size, np.linalg.norm(rounded - want) / size


@pytest.mark.parametrize("new", [3, 12, 64])
@pytest.mark.parametrize("qt", ["nf4", "fp4"])
def test_fp16_keeps_second_terms(new, qt):
    """Weights and scales of many different sizes, fp16: rounding weights or
    values to one fp16 term would be an error of 2^-10 / sqrt 12 of a term at
    most, 2.0e-4 on average, as large as the result's own rounding.  Allowed:
    the keys' NF4 values as one fp16 term (6.2e-5 of the score's spread, which
    is 1, so of the weights; none with FP4) and fp32 arithmetic."""
    L, hq, hk, dim = 2000, 16, 4, 128
    cache, table, K, V = filled(L, hk, dim, 32, "fp16", qt, 5 + new)
    q = torch.randn(new, hq, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(new)).to(torch.float16)
    got = attention_4bit(q, cache, table, i32([L]), cu_q=i32([0, new]), max_q=new, causal=False)
    qd = q.double().cpu().numpy()
    want = np.empty(qd.shape)
    for h in range(hq):
        s = qd[:, h] @ K[:, h // 4].T * dim ** -0.5
        p = np.exp(s - s.max(1, keepdims=True))
        want[:, h] = (p / p.sum(1, keepdims=True)) @ V[:, h // 4]
    err, u = norms(got, want, "fp16")
    assert err <= np.hypot(u, 1.2e-4 if qt == "nf4" else 8e-5), (err, u)


# --------------------------------------------------------------------------
@pytest.mark.parametrize("new", [1, 16, 64])
@pytest.mark.parametrize("dt,qt,bs", [("bf16", "nf4", 64), ("bf16", "nf4", 128), ("bf16", "fp4", 64), ("fp16", "nf4", 64)])
def test_cancelling_sums_do_not_drift(new, dt, qt, bs):
    """Uniform weights over 65536 normal rows, whose sum is 1/256 of their
    size: an error of the values with a mean would be 256 times as large in it.
    The kernel's own error: one fp16 rounding of a value by at most a unit of
    the last place (2^-10 / sqrt 6 of the value at most, 3e-4 on average) for
    bf16, second terms for fp16; fp32 sums of 65536 terms 2^-24 sqrt(65536) =
    1.5e-5 of the running sum."""
    L, dim = 65536, 128
    cache, table, _, V = filled(L, 1, dim, bs, dt, qt, new + bs)
    want = np.broadcast_to(V.mean(0), (new, 1, dim))
    assert np.linalg.norm(want) < 0.01 * np.sqrt(new * dim)
    q = torch.zeros(new, 1, dim, dtype=TDT[dt], device="cuda")
    got = attention_4bit(q, cache, table, i32([L]), cu_q=i32([0, new]), max_q=new, causal=False)
    err, u = norms(got, want, dt)
    assert err <= np.hypot(u, 5e-4 if dt == "bf16" else 5e-5), (err, u)


# --------------------------------------------------------------------------
@pytest.mark.parametrize("new", [[300], [12]])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,bs", [(64, 32), (128, 128), (256, 64)])
def test_a_large_key_leaves_rows_before_it_alone(new, dt, dim, bs):
    """Keys 2^20 times as large as their neighbours: hidden from the rows
    before them, whose scores are those of the small keys."""
    at = [300 - new[0] + 9, 299] if new[0] < 300 else [20, 100, 230, 299]

    def gain(n, isv):
        a = np.ones(n)
        if not isv:
            a *= 2.0 ** -10
            a[at] = 2.0 ** 10
        return a
    check([300], new, 4, 2, dim, bs, 16, dt, seed=dim, scale_gain=gain, scale=dim ** -0.5 * 2.0 ** 10)


@pytest.mark.parametrize("new", [[300], [12]])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_large_value_leaves_rows_before_it_alone(new, dt):
    at = [300 - new[0] + 9, 299] if new[0] < 300 else [20, 100, 230, 299]

    def gain(n, isv):
        a = np.ones(n)
        if isv:
            a *= 2.0 ** -10
            a[at] = 2.0 ** 10
        return a
    check([300], new, 4, 2, 64, 64, 16, dt, seed=64, scale_gain=gain)


# --------------------------------------------------------------------------
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("bits", ["inf", "nan"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("new,bad", [([4], 299), ([4], 297), ([12], 291), ([40], 270), ([300], 100), ([300], 290)])
def test_a_key_or_value_that_is_not_finite(new, bad, dt, bits, what):
    """Rows before such a key are as without it, and so are rows before such a
    value up to 48 rows of a cache head; elements outside the value's block are
    as they would be in every row."""
    lens, hq, hk, dim, bs = [300], 2, 2, 128, 64
    cache, table, K, V = make(lens, hk, dim, bs, 16, dt, "nf4", 77)
    page, at = int(table[0, bad // 16]), bad % 16
    scales = cache.k_scales if what == "k" else cache.v_scales
    scales[page, :, 0, at] = float(bits)           # of the first block of 64 elements
    q = torch.randn(new[0], hq, dim, generator=torch.Generator().manual_seed(3)).to(TDT[dt]).cuda()
    got = attention_4bit(q, cache, table, i32(lens), cu_q=i32([0] + new), max_q=new[0])
    got = got.double().cpu().numpy()
    pos = lens[0] - new[0] + np.arange(new[0])
    for h in range(hk):
        ref, bound = R.attend(q[:, h].double().cpu().numpy(), K[0][:, h], V[0][:, h], dim ** -0.5, np.zeros(new[0], int), pos + 1)
        ok = np.abs(got[:, h] - ref) <= 1.01 * (bound + R.U_OUT[dt] * np.abs(ref) + R.SUBNORMAL[dt])
        before = pos < bad
        if what == "k" or new[0] <= 48:
            assert ok[before].all()
        if what == "v":
            assert ok[:, 64:].all()
            assert not np.isfinite(got[~before, h, :64]).any()


# --------------------------------------------------------------------------
@pytest.mark.parametrize("lens,new,dim", [([300, 40], [1, 1], 128), ([300, 40], [9, 40], 128), ([300, 130], [90, 130], 64),
                                          ([300, 130], [3, 130], 256), ([300, 40], [5, 40], 32), ([9000], [1], 64)])
@pytest.mark.parametrize("dt,q_gain,k_gain", [("fp16", 2.0 ** 8, 2.0 ** 8), ("fp16", 2.0 ** 13, 2.0 ** 13), ("bf16", 2.0 ** 40, 2.0 ** 40),
                                              ("bf16", 2.0 ** 52, 2.0 ** 53)])
def test_large_scores_pick_one_key(lens, new, dim, dt, q_gain, k_gain):
    """Scores so far apart (2^20 and more) that the weights are one 1 and
    zeros: the result is the value of the best key, whatever its score's sign
    and size.  Rows whose best two keys are closer than the keys' rounding
    (6e-5 of the scores' size, taken tenfold) are left out."""
    cu = np.concatenate([[0], np.cumsum(new)])
    parts = [filled(n, 2, dim, 32, dt, "nf4", 7 + n, k_gain=k_gain, page=64) for n in lens]
    pages = [p[1].shape[1] for p in parts]
    cat = lambda name: torch.cat([getattr(p[0], name) for p in parts])
    cache = KVCache4bit.from_tensors(cat("k_codes"), cat("k_scales"), cat("v_codes"), cat("v_scales"))
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
    for b, p in enumerate(parts):
        table[b, :pages[b]] = p[1][0] + sum(pages[:b])
    q = (torch.randn(cu[-1], 4, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(dim)) * q_gain).to(TDT[dt])
    got = attention_4bit(q, cache, table, i32(lens), cu_q=i32(cu.tolist()), max_q=max(new)).double().cpu().numpy()
    qd = q.double().cpu().numpy()
    tested = negative = 0
    for b, n in enumerate(new):
        _, _, K, V = parts[b]
        for i in range(n):
            hi = lens[b] - n + i + 1
            for h in range(4):
                s = K[:hi, h // 2] @ qd[cu[b] + i, h]
                order = np.argsort(s)
                size = np.sqrt((K[:hi, h // 2] ** 2).sum(1).max() * (qd[cu[b] + i, h] ** 2).mean())
                if hi > 1 and s[order[-1]] - s[order[-2]] < 6e-4 * size:
                    continue
                want = V[order[-1], h // 2]
                have = got[cu[b] + i, h]
                # one fp16 rounding of the value and one of the result
                assert np.all(np.abs(have - want) <= (R.U_OUT[dt] + 2.0 ** -10) * np.abs(want) + R.SUBNORMAL[dt]), (b, i, h)
                tested += 1
                negative += s[order[-1]] < 0
    assert tested > 0.9 * 4 * cu[-1]
    assert negative > 0 or lens[-1] != new[-1]
