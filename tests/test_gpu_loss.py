"""cross_entropy_4bit and distill_4bit against float64 (tuning_reference)."""
import pytest
import torch

import quantized_matvec_amd as qmv
import tuning_reference as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def weight(V, K, bs=64, qt="nf4", dq=False, seed=0, dtype=BF, gain=2.0):
    g = torch.Generator().manual_seed(seed)
    packed, state = qmv.quantize_4bit((torch.randn(V, K, generator=g) * gain * K ** -0.5).to(dtype).cuda(), bs, qt, double_quant=dq)
    return packed, state, qmv.dequantize_4bit(packed, state, out_dtype=F32)


# The product's kernels round the weight T * a to 16 bits, except those for up
# to 64 rows, which round T alone (qmv_gemm.hip, qmv_gemv.hip, qmv_skinny.hip) and
# multiply by a in fp32.  Of FP4's values only 0, 1/4, 1/2 and 1 are the same in 16
# bits (1/6 is off by up to 2^-9 of itself in bf16).  So weights that are whole
# multiples of a power of two by their scale of 6 are exact from 65 rows on; below,
# a weight is off by up to the type's rounding, and the exact ones take those four values.
NARROW = 64
SAME_IN_16_BITS = [0, 3, 5, 7, 8, 11, 13, 15]


def whole_weight(V, K, bs=64, seed=0, table=False):
    """FP4 codes with scales of 6 * 2^-4: weights that are multiples of 2^-5 up to
    6 / 16, the same in every type, so that logits of small whole x are exact.
    With `table`, codes whose values are the same in 16 bits, scales of 2^-1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(256, (V * K // 2,), generator=g, device="cuda", dtype=torch.uint8)
    if table:
        t = torch.tensor(SAME_IN_16_BITS, device="cuda", dtype=torch.uint8)
        packed = t[(packed >> 4).int() % 8] << 4 | t[(packed & 15).int() % 8]
    state = qmv.QuantState((V, K), BF, bs, "fp4", absmax=torch.full((V * K // bs,), 0.5 if table else 6 / 16, device="cuda"))
    W = qmv.dequantize_4bit(packed, state, out_dtype=F32)
    assert torch.equal(W * 32, (W * 32).round()) and torch.equal(W, W.to(BF).float())
    return packed, state, W


def rows(T, K, dtype, seed=1, whole=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-2, 3, (T, K), generator=g) * (torch.rand(T, K, generator=g) < 0.5) if whole else torch.randn(T, K, generator=g)
    return x.to(dtype).cuda()


def targets(T, V, seed=2, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(V, (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = -100
    return t.cuda()


def dlosses(T, seed=3):
    return (torch.randn(T, generator=torch.Generator().manual_seed(seed)) * 3).cuda()


def teacher(T, V, k, dtype, seed=4):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, V, (T, k), generator=g)
    return ids.cuda(), (torch.randn(T, k, generator=g) * 3).to(dtype).cuda()


def exact(whole, T):
    return whole == "table" or (whole and T > NARROW)


def both(x, w, target, dloss, loss_dtype=F32, whole=False, what=""):
    packed, state, W = w
    whole = exact(whole, len(x))
    alone = qmv.cross_entropy_4bit(x, packed, state, target, loss_dtype=loss_dtype)
    loss, dx = qmv.cross_entropy_4bit(x, packed, state, target, dloss, loss_dtype=loss_dtype)
    R.check_loss(alone, None, x, W, target[:, None], exact_weights=whole, what=what + " alone")
    R.check_loss(loss, dx, x, W, target[:, None], dloss=dloss, exact_weights=whole, what=what)
    return loss, dx


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 33, 64, 65, 130, 448, 600])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("whole", [False, True, "table"])
def test_tokens(T, dtype, whole):
    V, K = 1000, 256
    w = whole_weight(V, K, table=whole == "table") if whole else weight(V, K, dq=T % 2 == 1, dtype=dtype)
    both(rows(T, K, dtype, whole=whole), w, targets(T, V), dlosses(T), whole=whole)


# fewer columns than a matrix-core tile, pieces and tails of the vocabulary
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 63, 255, 257, 4095, 8191, 8192, 8193, 8223, 16384, 20001])
@pytest.mark.parametrize("T,whole", [(3, True), (3, "table"), (40, True), (40, "table"), (300, True), (500, True)])
def test_vocabularies(V, T, whole):
    K = 128
    w = whole_weight(V, K, table=whole == "table")
    t = targets(T, V)
    t[0], t[1], t[2] = 0, V - 1, V  # the ends, and one past the end
    both(rows(T, K, BF, whole=True), w, t, dlosses(T), whole=whole)


@pytest.mark.parametrize("K,bs,qt,dq", [(32, 32, "nf4", True), (96, 32, "fp4", False), (320, 64, "nf4", True), (2048, 128, "nf4", True),
                                        (4096, 4096, "fp4", False), (1056, 32, "nf4", True)])
@pytest.mark.parametrize("T", [5, 100, 520])
def test_widths(K, bs, qt, dq, T):
    V = 777
    both(rows(T, K, BF), weight(V, K, bs, qt, dq), targets(T, V), dlosses(T))


# tokens in turns, pieces of the vocabulary where the tile product is not used (a width of 32)
@pytest.mark.parametrize("T,V,K", [(4500, 600, 64), (4000, 16400, 32), (5000, 300, 96)])
def test_turns_and_pieces(T, V, K):
    both(rows(T, K, BF, whole=True), whole_weight(V, K, bs=32), targets(T, V), dlosses(T), whole=True)


@pytest.mark.parametrize("T", [9, 300, 600])
def test_loss_types(T):
    for dtype in (BF, HF):
        w = weight(500, 128, dtype=dtype)
        both(rows(T, 128, dtype), w, targets(T, 500), dlosses(T), loss_dtype=dtype)


@pytest.mark.parametrize("T", [20, 520])
def test_no_target_counts(T):
    w = whole_weight(300, 64)
    t = torch.tensor([-1, 300, -2 ** 62, 2 ** 62] * (T // 4)).cuda()
    loss, dx = both(rows(T, 64, BF), w, t, dlosses(T))
    assert (loss == 0).all() and (dx == 0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,whole", [(6, True), (6, "table"), (70, True), (520, True)])
def test_certain_targets(dtype, T, whole):
    """A target far above all others: loss and 1 - q are tiny, not zero, and the
    others' part of the gradient is not flushed against the target's."""
    V, K = 900, 64
    w = whole_weight(V, K, bs=32, table=whole == "table")
    packed, state, _ = w
    packed.view(V, K // 2)[:, 0] = 0            # columns 0 and 1 are 0 ...
    packed.view(V, K // 2)[5, 0] = 0x70         # ... except in row 5
    W = qmv.dequantize_4bit(packed, state, out_dtype=F32)
    x = rows(T, K, dtype, whole=True) * (torch.rand(T, K, generator=torch.Generator().manual_seed(8)) < 0.1).cuda().to(dtype)
    x[:, 0] = torch.linspace(16, 64, T).round().to(dtype).cuda()  # row 5's logit is 6 to 24 above
    both(x, (packed, state, W), torch.full((T,), 5).cuda(), torch.full((T,), 8192.0 if dtype == HF else 1e4).cuda(), whole=whole)
    both(x, (packed, state, W), torch.full((T,), 6).cuda(), dlosses(T), whole=whole)


@pytest.mark.parametrize("T", [4, 300, 500])
def test_large_logits(T):
    """Logits in the thousands, and a maximum that moves from piece to piece."""
    V, K = 9000, 64
    packed, state, W = whole_weight(V, K)
    state.absmax.view(V, 1).mul_(torch.where(torch.arange(V) < 8192, 1.0, 64.0)[:, None].cuda())
    W = qmv.dequantize_4bit(packed, state, out_dtype=F32)
    both(rows(T, K, BF, whole=True) * 8, (packed, state, W), targets(T, V), dlosses(T), whole=True)
    state.absmax.view(V, 1).mul_(torch.where(torch.arange(V) < 8192, 64.0, 1.0 / 64)[:, None].cuda())
    W = qmv.dequantize_4bit(packed, state, out_dtype=F32)
    both(rows(T, K, BF, whole=True) * 8, (packed, state, W), targets(T, V), dlosses(T), whole=True)


@pytest.mark.parametrize("k", [1, 2, 8, 63, 64, 65, 128])
@pytest.mark.parametrize("T", [5, 66, 500])
@pytest.mark.parametrize("whole", [False, True, "table"])
def test_distill(k, T, whole):
    dtype = BF if k % 2 else HF
    V, K = 1234, 128
    w = whole_weight(V, K, table=whole == "table") if whole else weight(V, K, dtype=dtype)
    packed, state, W = w
    x, whole = rows(T, K, dtype, whole=whole), exact(whole, T)
    for tau, tt in ((1.0, F32), (2.0, BF), (0.5, HF)):
        ids, z = teacher(T, V, k, tt)
        g = dlosses(T)
        alone = qmv.distill_4bit(x, packed, state, ids, z, tau, loss_dtype=F32)
        loss, dx = qmv.distill_4bit(x, packed, state, ids, z, tau, g, loss_dtype=F32)
        R.check_loss(alone, None, x, W, ids, z, tau, exact_weights=whole)
        R.check_loss(loss, dx, x, W, ids, z, tau, g, exact_weights=whole)


@pytest.mark.parametrize("T,whole", [(8, True), (8, "table"), (504, True)])
def test_distill_rows_with_gaps(T, whole):
    """Ids that come twice, ids that are none, logits of -inf, rows without an entry, one entry of many."""
    V, K, k = 500, 64, 6
    packed, state, W = whole_weight(V, K, table=whole == "table")
    x = rows(T, K, BF, whole=True)
    inf = float("inf")
    ids = torch.tensor([[7, 7, 7, 7, 7, 7], [1, 2, 1, 2, 3, 1], [-1, 500, -5, 4, -1, -1], [-1] * 6, [9, 10, 11, 12, 13, 14],
                        [9, 10, 11, 12, 13, 14], [499, 498, 0, 499, -1, 0], [1, 2, 3, 4, 5, 6]])
    z = torch.tensor([[1.0, 2, 3, 4, 5, 6], [0.5, 1, -2, 3, 0, 0], [1, 2, 3, 4, 5, 6], [1, 2, 3, 4, 5, 6], [-inf, 1, -inf, 2, 0, -inf],
                      [-inf] * 6, [1, 1, 1, 1, 9, 1], [80, 0, 0, 0, 0, 0]])
    ids, z = ids.repeat(T // 8, 1).cuda(), z.repeat(T // 8, 1).cuda()
    g = dlosses(T)
    loss, dx = qmv.distill_4bit(x, packed, state, ids, z, 1.0, g, loss_dtype=F32)
    R.check_loss(loss, dx, x, W, ids, z, 1.0, g, exact_weights=exact(whole, T))
    assert (loss[3::8] == 0).all() and (loss[5::8] == 0).all() and (dx[3::8] == 0).all() and (dx[5::8] == 0).all()


@pytest.mark.parametrize("T,whole", [(8, "table"), (504, True)])
def test_distill_with_lowest_values(T, whole):
    """fp32's lowest value as a mask: it counts beside others of its kind, and not beside larger ones, at any temperature."""
    low = torch.finfo(F32).min
    V, K, tau = 300, 64, 0.5
    w = whole_weight(V, K, table=whole == "table")
    x = rows(T, K, BF, whole=True)
    z = torch.tensor([[low, low, low, low], [low, 1, 2, low], [low, low, low, 3], [0, low, -float("inf"), 0]] * (T // 4)).cuda()
    ids = torch.randint(V, (T, 4), generator=torch.Generator().manual_seed(2)).cuda()
    dl = dlosses(T)
    loss, dx = qmv.distill_4bit(x, w[0], w[1], ids, z, tau, dl, F32)
    # the bound takes the logits' size as that of the largest: lowest values as -inf, but where there is nothing else
    plain = torch.where((z == low).all(1, keepdim=True), 0.0, torch.where(z == low, -float("inf"), z))
    R.check_loss(loss, dx, x, w[2], ids, plain, tau, dl, exact(whole, T), "lowest")


def test_distill_of_one_certain_entry_is_cross_entropy():
    T, V, K = 60, 400, 128
    packed, state, W = weight(V, K)
    x, t, g = rows(T, K, BF), targets(T, V), dlosses(T)
    a, da = qmv.cross_entropy_4bit(x, packed, state, t, g, loss_dtype=F32)
    b, db = qmv.distill_4bit(x, packed, state, t[:, None], torch.full((T, 1), 3.0).cuda(), 1.0, g, loss_dtype=F32)
    R.check_loss(b, db, x, W, t[:, None], dloss=g)
    assert (a - b).abs().max() <= 2.0 ** -18 * (1 + a.abs().max())
    assert (da.float() - db.float()).abs().max() <= 2.0 ** -7 * da.float().abs().max()


def test_gradient_against_differences():
    """Whole weights and fp16 rows that move by 1/64: logits are exact in fp32, the
    loss is smooth, and the difference's error is its third derivative's."""
    T, V, K = 24, 300, 64
    packed, state, W = whole_weight(V, K)
    x, t = rows(T, K, HF, whole=True), targets(T, V, ignored=0.0)
    g = torch.Generator().manual_seed(6)
    d = torch.zeros(T, K)
    d[torch.arange(T), torch.randint(K, (T,), generator=g)] = 2.0 ** -6  # one element of each row
    d = d.to(HF).cuda()
    up, down = (qmv.cross_entropy_4bit(x + s * d, packed, state, t, loss_dtype=F32).double() for s in (1, -1))
    _, dx = qmv.cross_entropy_4bit(x, packed, state, t, torch.ones(T).cuda())
    h = 2.0 ** -6
    # |third derivative| <= 2 max|w|^3 per unit, losses off by 2^-20 of about 10, dx by a few parts of 2^-11
    bound = h * h / 6 * 2 * 0.375 ** 3 + 2 * 2.0 ** -20 * 16 / (2 * h) + 4 * 2.0 ** -11 * 0.75
    assert (((up - down) / (2 * h)) - (dx.double() * (d != 0)).sum(1)).abs().max() <= bound


def test_rows_that_are_not_finite_stay_alone():
    for T in (30, 600):
        packed, state, W = whole_weight(600, 128)
        x, t, g = rows(T, 128, BF, whole=True), targets(T, 600, ignored=0.0), dlosses(T)
        loss, dx = qmv.cross_entropy_4bit(x, packed, state, t, g)
        bad = x.clone()
        bad[3, 5], bad[9, 100] = float("nan"), float("inf")
        loss2, dx2 = qmv.cross_entropy_4bit(bad, packed, state, t, g)
        rest = [i for i in range(T) if i not in (3, 9)]
        assert torch.equal(loss[rest], loss2[rest]) and torch.equal(dx[rest], dx2[rest])
        assert not torch.isfinite(loss2[3])


def test_views_and_no_tokens():
    packed, state, W = whole_weight(200, 64)
    x, t, g = rows(12, 64, BF), targets(12, 200), dlosses(12)
    loss, dx = qmv.cross_entropy_4bit(x, packed, state, t, g)
    wide = torch.zeros(12, 3, 64, dtype=BF, device="cuda")
    wide[:, 2] = x
    loss2, dx2 = qmv.cross_entropy_4bit(wide[:, 2], packed, state, torch.stack((t, t), 1)[:, 1], torch.stack((g, g), 1)[:, 0])
    assert torch.equal(loss, loss2) and torch.equal(dx, dx2)
    out = torch.empty(12, 64, dtype=BF, device="cuda")
    assert qmv.cross_entropy_4bit(x, packed, state, t, g, dx=out)[1] is out and torch.equal(out, dx)
    assert qmv.cross_entropy_4bit(x[:0], packed, state, t[:0]).shape == (0,)
    loss, dx = qmv.distill_4bit(x[:0], packed, state, t[:0, None], g[:0, None], 1.0, g[:0])
    assert loss.shape == (0,) and dx.shape == (0, 64)


@pytest.mark.parametrize("T", [5, 90, 520])
def test_repeats_and_graphs(T):
    V, K = 9001, 128
    packed, state, W = weight(V, K, dq=True)
    x, t, g = rows(T, K, BF), targets(T, V), dlosses(T)
    ids, z = teacher(T, V, 9, F32)
    call = lambda: (*qmv.cross_entropy_4bit(x, packed, state, t, g), *qmv.distill_4bit(x, packed, state, ids, z, 1.0, g),
                    qmv.cross_entropy_4bit(x, packed, state, t))
    want = call()
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    x0, t0 = x.clone(), t.clone()
    for i in range(3):
        x.copy_(x0 if i != 1 else -x0)
        t.copy_(t0 if i != 1 else t0.flip(0))
        graph.replay()
        qmv.cross_entropy_4bit(x[:3], packed, state, t[:3], g[:3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_two_streams():
    packed, state, W = weight(5000, 256, dq=True)
    a = (rows(200, 256, BF), packed, state, targets(200, 5000), dlosses(200))
    b = (rows(200, 256, BF, seed=7), packed, state, targets(200, 5000, seed=8), dlosses(200))
    want = [qmv.cross_entropy_4bit(*c) for c in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(4):
        for i, (s, c) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i].append(qmv.cross_entropy_4bit(*c))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[i]))
