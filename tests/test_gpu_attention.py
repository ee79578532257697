"""attention_4bit on the GPU against the float64 form, per element within the
bound derived in kv_reference, over types, head layouts, head sizes, block
sizes, page sizes, query counts and masks."""
import numpy as np
import pytest
import torch

import kv_reference as R
from quantized_matvec_amd import KVCache4bit, attention_4bit, qmv

pytestmark = pytest.mark.gpu
TDT = {"fp16": torch.float16, "bf16": torch.bfloat16}
NAN16 = 0x7FFF                      # a NaN in both 16-bit types


def make(lens, hk, dim, bs, page, dt, qt, seed, spread=0.3, missing=(), spare=2, scale_gain=None):
    """A cache holding random rows of each sequence, its pages shuffled; every
    byte and scale that belongs to no token is garbage (NaN scales).  Returns
    the cache, the block table and the float64 rows [B][L, hk, D] (NaN rows
    where `missing` (b, page index) entries are left out of the table)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    width = max(max(need), 1)
    table = np.full((len(lens), width), -1, np.int32)
    kc = rng.integers(0, 256, (pages, hk, page, dim // 2)).astype(np.uint8)
    vc = rng.integers(0, 256, (pages, hk, page // 16, dim // 2, 16)).astype(np.uint8)
    ks = torch.full((pages, hk, dim // bs, page), NAN16, dtype=torch.int16).view(TDT[dt])
    vs = ks.clone()
    K, V = [], []
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        rows = []
        for codes, scales, isv in ((kc, ks, False), (vc, vs, True)):
            a = np.exp(rng.standard_normal((n, hk, dim // bs)) * spread)
            if scale_gain is not None:
                a = a * scale_gain(n, isv)[:, None, None]
            a = torch.from_numpy(a).to(TDT[dt])
            c = np.zeros((n, hk, dim // 2), np.uint8)
            for i in range(need[b]):
                lo, hi = i * page, min((i + 1) * page, n)
                pg = table[b, i]
                if isv:
                    c[lo:hi] = codes[pg].transpose(1, 3, 0, 2).reshape(page, hk, dim // 2)[:hi - lo]
                else:
                    c[lo:hi] = codes[pg].transpose(1, 0, 2)[:hi - lo]
                scales[pg, :, :, :hi - lo] = a[lo:hi].permute(1, 2, 0)
            rows.append(R.decode_rows(c, a.double().numpy(), qt))
        for (mb, mi) in missing:
            if mb == b:
                for r in rows:
                    r[mi * page:(mi + 1) * page] = np.nan
        K.append(rows[0])
        V.append(rows[1])
    for i, (mb, mi) in enumerate(missing):
        table[mb, mi] = -1 if i % 2 == 0 else pages + 7      # none, and out of range
    cache = KVCache4bit.from_tensors(torch.from_numpy(kc).cuda(), ks.cuda(), torch.from_numpy(vc).cuda(), vs.cuda(), qt)
    return cache, torch.from_numpy(table).cuda(), K, V


def check(lens, new, hq, hk, dim, bs, page, dt="bf16", qt="nf4", seed=0, causal=True, window=0, scale=None,
          missing=(), strided=False, use_max_kv=True, q_gain=1.0, scale_gain=None, max_q=None):
    cache, table, K, V = make(lens, hk, dim, bs, page, dt, qt, seed, missing=missing, scale_gain=scale_gain)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(new)
    x = (torch.randn(T, hq + 2 * hk, dim, generator=g) * q_gain).to(TDT[dt]).cuda()
    q = x[:, :hq] if strided else x[:, :hq].contiguous()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    single = all(n == 1 for n in new)
    out = None
    if strided:
        whole = torch.full((T, hq + 3, dim), 7.0, dtype=TDT[dt], device="cuda")
        out = whole[:, 2:2 + hq]
    got = attention_4bit(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         cu_q=None if single else torch.from_numpy(cu).cuda(), max_q=max_q or max(new),
                         max_kv=max(max(lens), 1) if use_max_kv else None, scale=scale, causal=causal,
                         window=window, out=out)
    torch.cuda.synchronize()
    if strided:
        assert got.data_ptr() == out.data_ptr()
        assert (whole[:, :2] == 7).all() and (whole[:, 2 + hq:] == 7).all()
    assert got.shape == (T, hq, dim) and got.dtype == TDT[dt]
    got = got.double().cpu().numpy()
    qd = q.double().cpu().numpy()
    G = hq // hk
    s = dim ** -0.5 if scale is None else scale
    for b, n in enumerate(new):
        pos = lens[b] - n + np.arange(n)
        hi = np.minimum(pos + 1, lens[b]) if causal else np.full(n, lens[b])
        lo = np.maximum(pos - window + 1, 0) if window else np.zeros(n, int)
        for h in range(hk):
            rows = qd[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, dim)
            ref, bound = R.attend(rows, K[b][:, h], V[b][:, h], s, np.repeat(lo, G), np.repeat(hi, G))
            bound = 1.01 * (bound + R.U_OUT[dt] * np.abs(ref) + R.SUBNORMAL[dt])
            have = got[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, dim)
            bad = np.argwhere(~(np.abs(have - ref) <= bound))
            assert bad.size == 0, (f"sequence {b} head {h}: {len(bad)} of {ref.size} outside, first {bad[:3].tolist()}: "
                                   f"got {have[tuple(bad[0])]}, want {ref[tuple(bad[0])]}, bound {bound[tuple(bad[0])]}")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("qt", ["nf4", "fp4"])
@pytest.mark.parametrize("dim,bs", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (160, 32),
                                    (192, 64), (224, 32), (256, 64), (256, 256)])
def test_decode_heads(dim, bs, dt, qt):
    check([1, 70, 333], [1, 1, 1], 8, 2, dim, bs, 16, dt, qt, seed=dim + bs)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (40, 1), (12, 4), (28, 4), (71, 1)])
def test_decode_groups(hq, hk):
    check([517, 40], [1, 1], hq, hk, 64, 64, 16, seed=hq)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
def test_lengths_and_pages(page):
    """Lengths around every page, tile and split border, empty sequences among them."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 0, 1023, 1025, 2047, 2300]
    check(lens, [1] * len(lens), 4, 2, 64, 32, page, seed=page, use_max_kv=page != 32)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [[2, 2], [3, 5], [1, 0, 9], [17, 33], [64, 1, 130], [200]])
def test_several_tokens(new, dt):
    check([n + 77 * (i + 1) for i, n in enumerate(new)], new, 8, 2, 128, 64, 16, dt, seed=sum(new))


@pytest.mark.parametrize("dim,bs", [(32, 32), (64, 32), (96, 32), (128, 32), (128, 64), (128, 128), (160, 32), (192, 32),
                                    (192, 64), (256, 32), (256, 64), (256, 128), (256, 256)])
@pytest.mark.parametrize("dt,qt", [("bf16", "nf4"), ("fp16", "fp4")])
def test_prompt_heads(dim, bs, dt, qt):
    check([150, 61], [150, 40], 4, 2, dim, bs, 32, dt, qt, seed=dim)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 1), (9, 3), (32, 2)])
def test_prompt_groups(hq, hk):
    check([301, 190], [301, 129], hq, hk, 64, 64, 64, seed=hq)


def test_prompt_over_a_long_past():
    check([3000], [130], 4, 1, 128, 64, 64, seed=3)
    check([5100, 4000], [20, 33], 8, 2, 64, 64, 16, "fp16", seed=4)


@pytest.mark.parametrize("window", [1, 2, 16, 50, 64, 100, 511])
@pytest.mark.parametrize("new", [[1, 1], [4, 3], [90, 140]])
def test_window(window, new):
    check([700, 150], new, 4, 2, 64, 64, 16, seed=window)
    check([700, 150], new, 4, 2, 64, 64, 16, seed=window, window=window)


@pytest.mark.parametrize("new", [[1, 1, 1], [5, 1, 2], [70, 100, 40]])
def test_not_causal(new):
    check([130, 400, 77], new, 4, 2, 128, 64, 16, seed=8, causal=False)


@pytest.mark.parametrize("new", [[5, 3], [40, 150]])
def test_more_tokens_than_the_cache_holds(new):
    """Tokens at negative positions see nothing: zeros, not NaN."""
    check([3, 0], new, 4, 2, 64, 32, 16, seed=9)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 90, 20]])
def test_missing_pages(new):
    """Pages without an entry, or with one out of range, hold no keys; a
    sequence without any page gives zeros."""
    check([200, 130, 40], new, 4, 2, 64, 64, 16, seed=10,
          missing=[(0, 0), (0, 3), (0, 4), (1, 5), (0, 12), (1, 8), (2, 0), (2, 1), (2, 2)])


@pytest.mark.parametrize("new", [[1, 1], [6, 70]])
def test_strided_operands(new):
    check([100, 300], new, 6, 2, 128, 64, 32, "fp16", seed=11, strided=True)


@pytest.mark.parametrize("new", [[1, 1], [40, 70]])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(new, scale):
    check([100, 300], new, 4, 2, 64, 64, 32, seed=12, scale=scale)


@pytest.mark.parametrize("new", [[1, 1], [40, 70]])
@pytest.mark.parametrize("q_gain,dt", [(2.0 ** -60, "bf16"), (2.0 ** 60, "bf16"), (2.0 ** -12, "fp16"), (30.0, "bf16")])
def test_query_magnitudes(q_gain, dt, new):
    """Queries far outside fp16's range (the scale brings the scores back)."""
    check([100, 300], new, 4, 2, 128, 64, 32, dt, seed=13, q_gain=q_gain, scale=0.1 / q_gain if q_gain != 30.0 else None)


@pytest.mark.parametrize("new", [[1], [50]])
@pytest.mark.parametrize("up", [False, True])
def test_value_magnitudes(new, up):
    """Value scales that grow (or shrink) by 2^60 along a sequence, keys of
    one magnitude: the weights times the scales leave fp16's range."""
    def gain(n, isv):
        e = np.linspace(-30, 30, n) if isv else np.zeros(n)
        return 2.0 ** (e if up else -e)
    check([700], new, 4, 2, 64, 64, 16, seed=14, scale_gain=gain)


@pytest.mark.parametrize("new", [[1], [60]])
def test_scores_that_grow(new):
    """Keys that grow along the sequence: the running maximum moves in every step."""
    def gain(n, isv):
        return np.ones(n) if isv else np.linspace(0.01, 12, n)
    check([900], new, 4, 2, 64, 64, 16, seed=15, scale_gain=gain)


def test_long_decode_is_split():
    check([40000], [1], 4, 1, 64, 64, 64, seed=16)
    check([30011, 12, 9000], [1, 1, 1], 8, 2, 64, 64, 64, "fp16", seed=17)


def test_max_q_below_the_tokens_leaves_the_others_alone():
    """Tokens past max_q are not worked on; nothing else is touched."""
    lens, new = [100, 80], [7, 3]
    cache, table, K, V = make(lens, 2, 64, 64, 16, "bf16", "nf4", 18)
    q = torch.randn(10, 4, 64, device="cuda").to(torch.bfloat16)
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 7, 10], dtype=torch.int32, device="cuda")
    full = attention_4bit(q, cache, table, kl, cu_q=cu, max_q=7)
    out = torch.full_like(q, 5.0)
    attention_4bit(q, cache, table, kl, cu_q=cu, max_q=3, out=out)
    torch.cuda.synchronize()
    assert (out[3:7] == 5).all()
    for a, b in ((0, 3), (7, 10)):
        assert torch.allclose(out[a:b].float(), full[a:b].float(), rtol=0.02, atol=0.01)


def test_garbage_lengths_and_offsets_stay_inside():
    """Lengths past the block table, negative ones and offsets outside the
    tokens are held to what is there."""
    cache, table, K, V = make([64, 64], 2, 64, 64, 16, "bf16", "nf4", 19)
    q = torch.randn(6, 4, 64, device="cuda").to(torch.bfloat16)
    for lens in ([2 ** 31 - 1, -5], [1 << 20, 64], [-2 ** 31, 2 ** 30]):
        kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for cu in ([0, 3, 6], [-4, 100, 9], [5, 2, 6], [0, 2 ** 31 - 1, -2 ** 31]):
            out = attention_4bit(q, cache, table, kl, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            assert out.shape == q.shape


def test_offsets_past_32_bits():
    """A cache whose codes take more than 2^32 bytes each; the pages used lie at its end."""
    page, hk, dim, bs = 1024, 8, 256, 256
    pages = (1 << 32) // (page * hk * dim // 2) + 6
    kc = torch.zeros(pages, hk, page, dim // 2, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(pages, hk, page // 16, dim // 2, 16, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pages, hk, 1, page, dtype=torch.bfloat16, device="cuda")
    vs = torch.zeros_like(ks)
    assert kc.numel() > 1 << 32
    small, table, K, V = make([1500], hk, dim, bs, page, "bf16", "nf4", 20, spare=0)
    n = small.num_pages
    for big, part in ((kc, small.k_codes), (vc, small.v_codes), (ks, small.k_scales), (vs, small.v_scales)):
        big[pages - n:] = part
    cache = KVCache4bit.from_tensors(kc, ks, vc, vs)
    q = torch.randn(40, 16, dim, device="cuda").to(torch.bfloat16)
    kl = torch.tensor([1500], dtype=torch.int32, device="cuda")
    for m in (1, 40):
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        want = attention_4bit(q[:m], small, table, kl, cu_q=cu, max_q=m)
        got = attention_4bit(q[:m], cache, table + (pages - n), kl, cu_q=cu, max_q=m)
        torch.cuda.synchronize()
        assert torch.equal(want, got)


def test_repeats_bit_for_bit_and_on_another_stream():
    cache, table, K, V = make([9000, 500], 2, 128, 64, 64, "bf16", "nf4", 21)
    kl = torch.tensor([9000, 500], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 16, 128, device="cuda").to(torch.bfloat16)
    want = attention_4bit(q, cache, table, kl)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        h = torch.randn(4096, 4096, device="cuda")
        for _ in range(30):
            h = torch.tanh(h @ h) * 0.01
        late = torch.zeros_like(q)
        late.copy_(q)                        # written by this stream, behind the products
        outs = [attention_4bit(late, cache, table, kl) for _ in range(5)]
    side.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_graph_replays():
    """Captured once, replayed with other queries and lengths between eager work."""
    cache, table, K, V = make([3000, 700, 90], 2, 128, 64, 16, "bf16", "nf4", 22)
    kl = torch.tensor([3000, 700, 90], dtype=torch.int32, device="cuda")
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    attention_4bit(q, cache, table, kl, max_kv=3000)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = attention_4bit(q, cache, table, kl, max_kv=3000)
    for r in range(4):
        q.copy_(torch.randn(3, 8, 128, device="cuda"))
        kl.copy_(torch.tensor([3000 - 700 * r, 700 - r, 90 - 30 * r], dtype=torch.int32))
        want = attention_4bit(q, cache, table, kl, max_kv=3000)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), r


def test_graphs_keep_their_own_workspace():
    """A captured call writes into memory of its graph: not into the workspace
    of the calls outside, and not into that of a graph that is gone."""
    from quantized_matvec_amd import attention
    cache, table, K, V = make([3000, 700], 2, 128, 64, 16, "bf16", "nf4", 27)
    kl = torch.tensor([3000, 700], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    want = attention_4bit(q, cache, table, kl, max_kv=3000)
    long = attention_4bit(q[:1], cache, table[:1], kl[:1], max_kv=3000)
    torch.cuda.synchronize()
    before = {k: w.data_ptr() for k, w in attention._WS.items()}
    graphs, outs = [], []
    for n in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attention_4bit(q[:n], cache, table[:n], kl[:n], max_kv=3000))
        graphs.append(g)
    assert {k: w.data_ptr() for k, w in attention._WS.items()} == before
    for r in range(3):
        for g, o, w in zip(graphs, outs, (long, want)):
            o.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w), r
        assert torch.equal(attention_4bit(q, cache, table, kl, max_kv=3000), want)
        torch.cuda.synchronize()


def test_refusals():
    cache, table, K, V = make([64], 2, 64, 64, 16, "bf16", "nf4", 23)
    kl = torch.tensor([64], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, cache=cache, block_table=table, kv_len=kl)
    attention_4bit(**ok)
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q[0]),
                dict(q=torch.cat([q, q])), dict(block_table=table.long()), dict(block_table=table.cpu()),
                dict(kv_len=kl.long()), dict(kv_len=torch.cat([kl, kl])), dict(cu_q=kl),
                dict(out=q.float()), dict(out=torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            attention_4bit(**{**ok, **bad})
    for bad in (dict(window=-1), dict(window=5, causal=False), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(qmv.QmvError):
            attention_4bit(**{**ok, **bad})
    torch.cuda.synchronize()


@pytest.mark.parametrize("dim,bs", [(64, 64), (128, 64), (256, 128)])
def test_many_sequences(dim, bs):
    """More sequences than a workgroup has threads, many of them empty or without tokens."""
    rng = np.random.default_rng(dim)
    lens = rng.integers(0, 40, 900)
    lens[rng.integers(0, 900, 200)] = 0
    check(lens.tolist(), [1] * 900, 2, 1, dim, bs, 16, seed=dim)
    new = rng.integers(0, 3, 900)
    new[:300] = 0
    new[899] = 2
    check((lens + new).tolist(), new.tolist(), 2, 1, dim, bs, 16, "fp16", seed=dim + 1)


@pytest.mark.parametrize("hq,hk,new", [(8, 8, [17, 33, 48]), (64, 4, [2, 1, 3]), (34, 2, [2, 0, 1]), (6, 2, [1, 16, 15]),
                                       (24, 1, [1, 1, 1]), (40, 1, [1, 1, 1]), (2, 2, [47, 1, 32])])
@pytest.mark.parametrize("dim,dt", [(64, "fp16"), (96, "bf16"), (128, "bf16"), (256, "fp16")])
def test_row_tiles(hq, hk, new, dim, dt):
    """17 to 48 rows of a cache head: tiles that end inside a token, that a
    sequence fills in part or not at all, over short and divided sequences."""
    check([70, 900, 3000], new, hq, hk, dim, 32, 16, dt, seed=hq + dim)
    check([5000, 49, 0], new, hq, hk, dim, 32, 64, dt, "fp4", seed=hq + dim + 1, window=100)
    check([48, 47, 260], new, hq, hk, dim, 32, 16, dt, seed=hq + dim + 2, causal=False, missing=[(2, 1)], strided=True)


def test_uneven_batch_over_every_division():
    """Sequences whose steps fall on all sides of the division among waves and workgroups."""
    lens = [9000, 1, 64, 700, 12000, 65, 3, 4097, 0, 511]
    check(lens, [1] * 10, 8, 2, 128, 64, 64, seed=31)
    check(lens, [1] * 10, 32, 4, 64, 32, 16, "fp16", "fp4", seed=32)
    check(lens, [1] * 10, 2, 1, 256, 64, 32, seed=33)


def test_long_sums_do_not_drift():
    """Uniform weights over 60000 values of one block scale: the values cancel,
    their rounding must not add up.  The sum of N values of variance s^2 is of
    size s sqrt(N), so a bias of 6e-5 of a value (the fp16 rounding of the NF4
    values) would be 1.5 % of it; the result's own rounding is 2^-9."""
    for dt, tol in (("bf16", 2.5e-3), ("fp16", 3.5e-4)):
        for new in ([1], [24]):
            cache, table, K, V = make([60000], 1, 128, 64, 64, dt, "nf4", 41, spread=0.0)
            q = torch.zeros(new[0], 4, 128, dtype=TDT[dt], device="cuda")
            kl = torch.tensor([60000], dtype=torch.int32, device="cuda")
            cu = torch.tensor([0, new[0]], dtype=torch.int32, device="cuda")
            got = attention_4bit(q, cache, table, kl, cu_q=cu, max_q=new[0], causal=False).double().cpu().numpy()
            want = V[0][:, 0].mean(0)
            err = np.linalg.norm(got - want) / np.linalg.norm(np.broadcast_to(want, got.shape))
            assert err <= tol, (dt, new, err)
