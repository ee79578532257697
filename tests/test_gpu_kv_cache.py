"""rotary, kv_append_4bit and kv_dequantize_4bit on the GPU.

rotary is pinned bit for bit: its definition rounds every product and sum in
fp32 and the result once.  The append is pinned bit for bit against the
codec's oracle on the rotated, rounded rows, and the read-back against the
oracle's dequantization."""
import numpy as np
import pytest
import torch

import kv_reference as R
import oracle as O
from quantized_matvec_amd import (KVCache4bit, kv_append_4bit, kv_dequantize_4bit, qmv, rope_frequencies, rope_table, rotary,
                                  rotary_backward)

pytestmark = pytest.mark.gpu
TDT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16).numpy()


def rounded(x, dt):
    """float32 values -> their bits in dt (round to nearest even), by torch on the CPU."""
    return bits(torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TDT[dt]))


def rows(T, heads, dim, dt, seed, strided):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, sum(heads), dim, generator=g).to(TDT[dt]).cuda()
    parts = list(x.split(heads, 1))
    return parts if strided else [p.contiguous() for p in parts]


# --------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 64), (128, 2), (96, 24), (96, 36), (80, 80), (40, 14), (8, 8),
                                     (256, 192), (32, 10)])
def test_rotary_bits(dim, rot, interleaved, dt):
    T, hq, hk = 37, 5, 2
    q, k = rows(T, [hq, hk], dim, dt, dim + rot, strided=rot % 4 == 0)
    table = rope_table(rope_frequencies(rot), 500)
    tab = table.cpu().numpy()
    pos = torch.from_numpy(np.random.default_rng(rot).integers(0, 500, T))
    pos[3], pos[7], pos[9] = -1, 500, 1 << 40             # outside: zero rows
    for fn, inverse in ((rotary, False), (rotary_backward, True)):
        outs = fn(q, k, table, pos.cuda(), interleaved=interleaved)
        torch.cuda.synchronize()
        for x, y in zip((q, k), outs):
            want = R.rotate(x.float().cpu().numpy(), tab, pos.tolist(), interleaved, inverse, np.float32)
            assert np.array_equal(bits(y), rounded(want, dt))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 24), (64, 18)])
def test_rotary_in_place_and_strided_outputs(dim, rot, interleaved):
    T = 131
    table = rope_table(rope_frequencies(rot), 200)
    pos = torch.arange(T, device="cuda")
    q, k = rows(T, [6, 2], dim, "bf16", 5, strided=True)
    want_q, want_k = rotary(q.contiguous(), k.contiguous(), table, pos, interleaved=interleaved)
    whole = torch.full((T, 11, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    got, _ = rotary(q, None, table, pos, interleaved=interleaved, q_out=whole[:, 1:7])
    a, b = rotary(q, k, table, pos, interleaved=interleaved, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert a.data_ptr() == q.data_ptr() and torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(got, want_q) and (whole[:, 0] == 3).all() and (whole[:, 7:] == 3).all()


def test_rotary_lengths():
    table = rope_table(rope_frequencies(64), 4096)
    for T in (0, 1, 2, 63, 64, 65, 4096):
        q, = rows(T, [3], 64, "bf16", T, strided=False)
        pos = torch.arange(T, device="cuda").flip(0).contiguous()
        y, none = rotary(q, None, table, pos)
        torch.cuda.synchronize()
        assert none is None
        want = R.rotate(q.float().cpu().numpy(), table.cpu().numpy(), pos.tolist(), False, False, np.float32)
        assert np.array_equal(bits(y), rounded(want, "bf16"))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_backward_is_the_adjoint_and_the_difference_quotient(interleaved):
    """<dY, J x'> = <J^T dY, x'> for the linear map, and central differences of
    a loss, in fp32 (a relative 2^-24 for each product and sum: 1e-5 over the
    4000 terms with room)."""
    T, H, D, rot = 9, 4, 64, 48
    table = rope_table(rope_frequencies(rot), 64, gain=1.3)
    pos = torch.arange(T, device="cuda") * 7
    x, dy, d = (rows(T, [H], D, "fp32", s, False)[0] for s in (1, 2, 3))
    dx, _ = rotary_backward(dy, None, table, pos, interleaved=interleaved)
    jd, _ = rotary(d, None, table, pos, interleaved=interleaved)
    dot = lambda a, b: float((a.double() * b.double()).sum())
    size = float(dy.double().norm() * d.double().norm())
    assert abs(dot(dy, jd) - dot(dx, d)) <= 1e-5 * size
    eps = 2.0 ** -3
    up, _ = rotary(x + eps * d, None, table, pos, interleaved=interleaved)
    down, _ = rotary(x - eps * d, None, table, pos, interleaved=interleaved)
    assert abs(dot(dy, (up.double() - down.double()) / (2 * eps)) - dot(dx, d)) <= 1e-5 * size


def test_rope_tables():
    """cos and sin rounded once from float64, at positions where fp32 angles would be wrong."""
    for rot, theta, n in ((128, 10000.0, 1000), (64, 500000.0, 131072), (2, 10000.0, 5)):
        f = rope_frequencies(rot, theta)
        got = rope_table(f, n, gain=1.25).cpu().numpy().astype(np.float64)
        a = np.arange(n, dtype=np.float64)[:, None] * np.asarray(f)
        want = 1.25 * np.stack([np.cos(a), np.sin(a)], -1)
        # one fp32 rounding, float64 angles and their cos and sin to a few ulps
        assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1e-14 * (1 + a[..., None]))


# --------------------------------------------------------------------------
def build_table(lens, page, seed, spare=3):
    need = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def check_append(lens, new, hq, hk, dim, bs, page, dt="bf16", qt="nf4", rot=None, interleaved=False, strided=False, seed=0,
                 max_pos=None, data=None):
    T = sum(new)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, pages = build_table(lens, page, seed)
    cache = KVCache4bit(pages, hk, page, dim, bs, qt, TDT[dt])
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0xA5)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(-3.0)
    before = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]
    q, k, v = rows(T, [hq, hk, hk], dim, dt, seed, strided)
    if data is not None:
        k, v = data(k), data(v)
    rope = None if rot is None else rope_table(rope_frequencies(rot), max_pos or max(lens))
    single = all(n == 1 for n in new)
    bt, kl = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    cud = None if single else torch.from_numpy(cu).cuda()
    got_q = kv_append_4bit(cache, k, v, bt, kl, cu_q=cud, max_q=max(new), q=None if rot is None else q, table=rope,
                           interleaved=interleaved)
    back = kv_dequantize_4bit(cache, bt, kl, T, cu_q=cud, max_q=max(new))
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)])
    kk = k.float().cpu().numpy()
    if rot is not None:
        tab = rope.cpu().numpy()
        want = R.rotate(q.float().cpu().numpy(), tab, pos, interleaved, False, np.float32)
        assert np.array_equal(bits(got_q), rounded(want, dt))
        kk = R.rotate(kk, tab, pos, interleaved, False, np.float32)
    kk = torch.from_numpy(np.ascontiguousarray(kk, np.float32)).to(TDT[dt])
    seq = np.repeat(np.arange(len(lens)), new)
    pg, at = table[seq, pos // page], pos % page
    have = [t.cpu() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]
    touched = [torch.zeros(t.shape, dtype=torch.bool) for t in have]
    for name, x, codes, scales, ci, si in (("k", kk, have[0], have[2], 0, 2), ("v", v.cpu(), have[1], have[3], 1, 3)):
        c_ref, a_ref = R.encode_rows(x.double().numpy(), bs, qt)
        if name == "v":
            c_got = codes.numpy()[pg, :, at // 16, :, at % 16]
            touched[ci][pg, :, at // 16, :, at % 16] = True
        else:
            c_got = codes.numpy()[pg, :, at]
            touched[ci][pg, :, at] = True
        a_got = scales.double().numpy()[pg, :, :, at]
        touched[si][pg, :, :, at] = True
        assert np.array_equal(a_got, a_ref), name
        assert np.array_equal(c_got, c_ref), (name, np.argwhere(c_got != c_ref)[:4])
        # fp32(T a) rounded to the type
        t32 = np.stack([O.code_table(qt)[c_ref >> 4], O.code_table(qt)[c_ref & 15]], -1).reshape(x.shape)
        vals = (t32.reshape(a_ref.shape + (-1,)) * a_ref.astype(np.float32)[..., None]).astype(np.float32).reshape(x.shape)
        assert np.array_equal(bits(back[0 if name == "k" else 1]), rounded(vals, dt)), name
    for b, h, t in zip(before, have, touched):               # nothing else was written
        assert torch.equal(b.cpu()[~t], h[~t])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("qt", ["nf4", "fp4"])
@pytest.mark.parametrize("dim,bs", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (160, 32),
                                    (192, 64), (224, 32), (256, 128), (256, 256)])
def test_append_bits(dim, bs, dt, qt):
    check_append([20, 1, 67], [1, 1, 1], 4, 2, dim, bs, 16, dt, qt, rot=dim, seed=dim + bs)
    check_append([20, 3, 67], [20, 2, 33], 4, 2, dim, bs, 16, dt, qt, rot=dim, seed=dim + bs + 1, strided=True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [None, 2, 10, 24, 32, 64, 96])
def test_append_partial_rotation(rot, interleaved):
    check_append([40, 90], [40, 21], 3, 1, 96, 32, 32, rot=rot, interleaved=interleaved, seed=7)


@pytest.mark.parametrize("page", [16, 32, 64, 1024])
def test_append_borders(page):
    """Chunks that begin and end anywhere in a page and in a group of 16 tokens."""
    lens = [1, 15, 16, 17, 31, 33, 64, 100, 0, 130, 2000]
    new = [1, 3, 16, 17, 15, 1, 64, 37, 0, 129, 500]
    check_append(lens, new, 2, 2, 64, 32, page, rot=64, seed=page)


def test_append_more_rows_than_a_workgroup():
    check_append([700] * 3, [700, 1, 350], 32, 8, 128, 64, 64, rot=128, seed=3, strided=True)


@pytest.mark.parametrize("qt", ["nf4", "fp4"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_hard_values(dt, qt):
    """Zero rows, constant rows, tiny and huge rows, every significand, exact midpoints of the FP4 table."""
    def data(x):
        x = x.clone()
        x[0] = 0
        x[1] = 1.5
        x[2] *= 2.0 ** -100 if dt == "bf16" else 2.0 ** -12
        x[3] *= 2.0 ** 100 if dt == "bf16" else 2.0 ** 12
        x[4, :, 1:] = 0
        x[5] *= 2.0 ** -125 if dt == "bf16" else 2.0 ** -20
        x[6] = torch.arange(x[6].numel(), device="cuda").view_as(x[6]).to(x.dtype) / 256
        x[7] = torch.linspace(-1, 1, x.shape[2], device="cuda").to(x.dtype)
        x[8] = torch.tensor([0, 1, 3, 5, 7, 10, 14, 20, 24, -1, -3, -5, -7, -10, -14, -20], device="cuda").repeat(4).to(x.dtype) / 24
        return x
    check_append([40], [40], 2, 2, 64, 32, 16, dt, qt, seed=4, data=data)
    check_append([40], [40], 2, 2, 64, 64, 16, dt, qt, seed=5, data=data)


def test_append_past_the_rope_table_is_zero():
    table, pages = build_table([40], 16, 1)
    cache = KVCache4bit(pages, 2, 16, 64, 32)
    q, k, v = rows(40, [4, 2, 2], 64, "bf16", 1, False)
    rope = rope_table(rope_frequencies(64), 30)
    bt, kl = torch.from_numpy(table).cuda(), torch.tensor([40], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    qo = kv_append_4bit(cache, k, v, bt, kl, cu_q=cu, q=q, table=rope)
    kb, vb = kv_dequantize_4bit(cache, bt, kl, 40, cu_q=cu)
    torch.cuda.synchronize()
    assert (qo[30:] == 0).all() and (kb[30:] == 0).all()
    assert (qo[:30] != 0).any() and (vb[30:] != 0).any()


def test_append_skips_tokens_without_a_page():
    """Missing and out-of-range pages, positions past the block table and
    negative ones are not written and read back as zeros; queries are turned."""
    cache = KVCache4bit(4, 2, 16, 64, 32)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x5A)
    bt = torch.tensor([[1, -1, 9], [2, 3, -2 ** 31]], dtype=torch.int32, device="cuda")
    kl = torch.tensor([60, 10], dtype=torch.int32, device="cuda")   # 60 > 3 pages of 16; 10 < its 14 tokens
    cu = torch.tensor([0, 60, 74], dtype=torch.int32, device="cuda")
    q, k, v = rows(74, [4, 2, 2], 64, "bf16", 2, False)
    rope = rope_table(rope_frequencies(64), 64)
    qo = kv_append_4bit(cache, k, v, bt, kl, cu_q=cu, max_q=60, q=q, table=rope)
    kb, vb = kv_dequantize_4bit(cache, bt, kl, 74, cu_q=cu, max_q=60)
    torch.cuda.synchronize()
    assert (kb[16:60] == 0).all() and (vb[16:60] == 0).all() and (vb[60:64] == 0).all()
    assert (vb[:16].abs().amax((1, 2)) > 0).all() and (vb[64:].abs().amax((1, 2)) > 0).all()
    assert (cache.k_codes[0] == 0x5A).all() and (cache.k_codes[3] == 0x5A).all()
    assert (cache.k_codes[2, :, 10:] == 0x5A).all()
    want = R.rotate(q.float().cpu().numpy(), rope.cpu().numpy(), list(range(60)) + list(range(-4, 10)), False, False, np.float32)
    assert np.array_equal(bits(qo), rounded(want, "bf16"))


def test_append_garbage_lengths_and_offsets_stay_inside():
    cache = KVCache4bit(4, 2, 16, 64, 32)
    bt = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    q, k, v = rows(6, [4, 2, 2], 64, "bf16", 2, False)
    rope = rope_table(rope_frequencies(64), 64)
    for lens in ([2 ** 31 - 1, -5], [1 << 20, 32], [-2 ** 31, 2 ** 30]):
        kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for cu in ([0, 3, 6], [-4, 100, 9], [5, 2, 6], [0, 2 ** 31 - 1, -2 ** 31]):
            c = torch.tensor(cu, dtype=torch.int32, device="cuda")
            kv_append_4bit(cache, k, v, bt, kl, cu_q=c, q=q, table=rope)
            kv_dequantize_4bit(cache, bt, kl, 6, cu_q=c)
            torch.cuda.synchronize()


def test_append_in_place_queries_and_composition():
    """The append holds what rotary and quantize_4bit give one after the other."""
    T, hq, hk, dim, bs = 50, 8, 2, 128, 64
    q, k, v = rows(T, [hq, hk, hk], dim, "bf16", 6, True)
    rope = rope_table(rope_frequencies(dim), T)
    pos = torch.arange(T, device="cuda")
    rq, rk = rotary(q, k, rope, pos)
    cache = KVCache4bit(4, hk, 16, dim, bs)
    bt = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    kl, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([T], [0, T]))
    out = kv_append_4bit(cache, k, v, bt, kl, cu_q=cu, q=q, table=rope, q_out=q)
    assert out.data_ptr() == q.data_ptr() and torch.equal(q, rq)
    back = kv_dequantize_4bit(cache, bt, kl, T, cu_q=cu)
    for x, got in ((rk, back[0]), (v, back[1])):
        packed, st = qmv.quantize_4bit(x.contiguous(), bs, "nf4")
        assert torch.equal(qmv.dequantize_4bit(packed, st, out_dtype=torch.bfloat16).view_as(got), got)


def test_graph_replays():
    cache = KVCache4bit(8, 2, 16, 64, 32)
    bt = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    kl = torch.tensor([5, 30], dtype=torch.int32, device="cuda")
    q, k, v = (x.clone() for x in rows(2, [4, 2, 2], 64, "bf16", 8, False))
    rope = rope_table(rope_frequencies(64), 64)
    kv_append_4bit(cache, k, v, bt, kl, q=q, table=rope)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kv_append_4bit(cache, k, v, bt, kl, q=q, table=rope)
        kb, vb = kv_dequantize_4bit(cache, bt, kl, 2)
    for r in range(4):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        kl.add_(7)
        want = kv_append_4bit(cache, k, v, bt, kl, q=q, table=rope)
        wk, wv = kv_dequantize_4bit(cache, bt, kl, 2)
        torch.cuda.synchronize()
        for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kb, wk) and torch.equal(vb, wv), r


def test_refusals():
    cache = KVCache4bit(4, 2, 16, 64, 32)
    bt = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    kl = torch.tensor([1], dtype=torch.int32, device="cuda")
    q, k, v = rows(1, [4, 2, 2], 64, "bf16", 9, False)
    rope = rope_table(rope_frequencies(64), 64)
    ok = dict(cache=cache, k=k, v=v, block_table=bt, kv_len=kl, q=q, table=rope)
    kv_append_4bit(**ok)
    for bad in (dict(k=k.half()), dict(v=v[:, :1]), dict(k=k[..., :32]), dict(v=v.cpu()), dict(q=q.float()), dict(table=None),
                dict(table=rope.double()), dict(table=rope.cpu()), dict(table=rope[:, :, 0]), dict(kv_len=kl.cpu()),
                dict(block_table=bt[0]), dict(q=q[..., :32]), dict(q=None, q_out=q), dict(cu_q=kl)):
        with pytest.raises(ValueError):
            kv_append_4bit(**{**ok, **bad})
    with pytest.raises(qmv.QmvError):                     # more is rotated than a head has
        kv_append_4bit(**{**ok, "table": rope_table(rope_frequencies(96), 8)})
    with pytest.raises(qmv.QmvError):
        kv_append_4bit(**{**ok, "cu_q": torch.tensor([0, 1], dtype=torch.int32, device="cuda"), "max_q": 0})
    for args in ((4, 2, 24, 64, 32), (4, 2, 48, 64, 32)):  # page sizes
        with pytest.raises((ValueError, qmv.QmvError)):
            c = KVCache4bit(*args)
            kv_append_4bit(**{**ok, "cache": c})
    c = KVCache4bit(4, 2, 16, 64, 32, dtype=torch.float32)
    with pytest.raises(qmv.QmvError):
        kv_append_4bit(**{**ok, "cache": c, "k": k.float(), "v": v.float(), "q": q.float()})
    with pytest.raises(ValueError):
        rotary(q, k, rope, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        rotary(q, k, rope, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        rotary(q, k.float(), rope, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        rotary(q, k, rope, torch.zeros(1, dtype=torch.int64, device="cuda"), q_out=q.float())
    torch.cuda.synchronize()


@pytest.mark.parametrize("interleaved,rot", [(False, 128), (True, 64), (False, 24)])
def test_rotary_of_many_tokens_is_that_of_its_parts(interleaved, rot):
    """A call large enough for several heads a thread, bit for bit against small calls."""
    T = 50000 if rot == 128 else 20000
    table = rope_table(rope_frequencies(rot), 4096)
    q, k = rows(T, [7, 2], 128, "bf16", 3, strided=True)
    pos = torch.arange(T, device="cuda") % 4100
    yq, yk = rotary(q, k, table, pos, interleaved=interleaved)
    for a in (0, 777, T // 2, T - 100):
        pq, pk = rotary(q[a:a + 100], k[a:a + 100], table, pos[a:a + 100].contiguous(), interleaved=interleaved)
        torch.cuda.synchronize()
        assert torch.equal(yq[a:a + 100], pq) and torch.equal(yk[a:a + 100], pk), a


@pytest.mark.parametrize("dim,bs,hk", [(128, 64, 8), (64, 32, 3), (256, 64, 2), (96, 32, 5)])
def test_append_of_many_tokens_is_that_of_its_parts(dim, bs, hk):
    """Long calls (several rows a thread, groups of 16 positions) against the
    same tokens appended a few at a time: the cache's bytes are the same."""
    T, past, hq = 4000, 5, 2 * hk
    pages = -(-(T + past) // 64)
    bt = torch.randperm(pages, device="cuda").to(torch.int32)[None]
    q, k, v = rows(T, [hq, hk, hk], dim, "bf16", dim, strided=True)
    rope = rope_table(rope_frequencies(dim), T + past)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    one, many = KVCache4bit(pages, hk, 64, dim, bs), KVCache4bit(pages, hk, 64, dim, bs)
    got = kv_append_4bit(one, k, v, bt, i32([past + T]), cu_q=i32([0, T]), q=q, table=rope)
    back = kv_dequantize_4bit(one, bt, i32([past + T]), T, cu_q=i32([0, T]))
    at, parts, reads = 0, [], []
    sizes = [1, 6, 7, 8, 9, 100, 333]
    while at < T:
        n = min(sizes[len(parts) % len(sizes)], T - at)
        lens, cu = i32([past + at + n]), i32([0, n])
        parts.append(kv_append_4bit(many, k[at:at + n], v[at:at + n], bt, lens, cu_q=cu, q=q[at:at + n], table=rope))
        reads.append(kv_dequantize_4bit(many, bt, lens, n, cu_q=cu))
        at += n
    torch.cuda.synchronize()
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, name), getattr(many, name)), name
    assert torch.equal(got, torch.cat(parts))
    for x in (0, 1):
        assert torch.equal(back[x], torch.cat([r[x] for r in reads]))


def test_dequantize_into_given_strided_outputs():
    cache = KVCache4bit(4, 2, 16, 64, 32)
    bt = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    q, k, v = rows(40, [4, 2, 2], 64, "bf16", 12, True)
    kl, cu = torch.tensor([40], dtype=torch.int32, device="cuda"), torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    kv_append_4bit(cache, k, v, bt, kl, cu_q=cu)
    want = kv_dequantize_4bit(cache, bt, kl, 40, cu_q=cu)
    whole = torch.full((40, 7, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    kv_dequantize_4bit(cache, bt, kl, 40, cu_q=cu, k_out=whole[:, 1:3], v_out=whole[:, 4:6])
    torch.cuda.synchronize()
    assert torch.equal(whole[:, 1:3], want[0]) and torch.equal(whole[:, 4:6], want[1])
    assert (whole[:, [0, 3, 6]] == 9).all()
