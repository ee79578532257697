"""lora_4bit and lora_4bit_backward against float64 (tuning_reference), at the
sizes where the kernels divide their work and at uses that a caller may make."""
import pytest
import torch

import quantized_matvec_amd as qmv
import tuning_reference as R

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def weight(N, K, bs=64, qt="nf4", dq=False, seed=0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    packed, state = qmv.quantize_4bit((torch.randn(N, K, generator=g) * K ** -0.5).to(dtype).cuda(), bs, qt, double_quant=dq)
    return packed, state, qmv.dequantize_4bit(packed, state, out_dtype=torch.float32)


def case(T, N, K, n, rank, dtype, index=None, seed=1, bs=64, qt="nf4", dq=False):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, gain=1.0: (torch.randn(*s, generator=g) * gain).to(dtype).cuda()
    packed, state, W = weight(N, K, bs, qt, dq, seed + 100, dtype)
    down, up = rnd(n, rank, K, gain=K ** -0.5), rnd(n, N, rank, gain=0.5 * rank ** -0.5)
    scale = (0.5 + torch.rand(n, generator=g)).cuda()
    if index is None:
        index = torch.randint(-1, n, (T,), generator=g)
    return dict(x=rnd(T, K), dy=rnd(T, N, gain=0.1), packed=packed, state=state, W=W, down=down, up=up, scale=scale,
                index=torch.as_tensor(index, dtype=torch.int32).cuda(), adapters=qmv.LoraAdapters(down, up, scale))


def forward(c, **kw):
    return qmv.lora_4bit(c["x"], c["packed"], c["state"], c["adapters"], c["index"], **kw)


def backward(c, **kw):
    return qmv.lora_4bit_backward(c["dy"], c["x"], c["packed"], c["state"], c["adapters"], c["index"], **kw)


def check_forward(c, y, bias=None, what="y"):
    R.check_lora(y, c["x"], c["W"], c["down"], c["up"], c["scale"], c["index"], bias, what)


def check_backward(c, grads, what=""):
    R.check_lora_backward(grads, c["dy"], c["x"], c["W"], c["down"], c["up"], c["scale"], c["index"], what)


# tokens on both sides of every rule that picks a kernel or a division
TOKENS = [1, 2, 8, 9, 16, 17, 33, 64, 65, 127, 200, 447, 448, 513]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tokens(T, dtype):
    c = case(T, 352, 320, 3, 16, dtype, dq=T % 2 == 0)
    check_forward(c, forward(c))
    check_backward(c, backward(c))


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 120, 128])
@pytest.mark.parametrize("T", [3, 70, 520])
def test_ranks(T, rank):
    c = case(T, 288, 512, 4, rank, BF if rank % 16 else HF)
    check_forward(c, forward(c, out_dtype=torch.float32))
    check_backward(c, backward(c, grad_dtype=torch.float32))


@pytest.mark.parametrize("N,K,bs,qt", [(32, 32, 32, "nf4"), (64, 96, 32, "fp4"), (544, 1056, 32, "nf4"), (96, 4096, 4096, "fp4"),
                                       (1024, 128, 128, "nf4"), (416, 2304, 256, "fp4")])
@pytest.mark.parametrize("T", [1, 40, 300, 700])
def test_shapes(N, K, bs, qt, T):
    c = case(T, N, K, 2, 16, BF, bs=bs, qt=qt, dq=bs < 128)
    bias = torch.randn(N).to(BF).cuda()
    check_forward(c, forward(c, bias=bias), bias)
    check_backward(c, backward(c))


@pytest.mark.parametrize("N,K", [(1, 64), (33, 64), (257, 320), (1000, 32)])
@pytest.mark.parametrize("T", [1, 20, 600])
def test_odd_widths_forward(N, K, T):
    c = case(T, N, K, 3, 8, HF, bs=32)
    check_forward(c, forward(c))


# enough tokens and columns for the tile product (640 tokens, 144 tiles of 256 x 256), whole tiles and
# parts of them, of the outputs (forward: N, backward: K) or sums; turns of 8192 and of 4096 tokens
@pytest.mark.parametrize("T,N,K,rank", [(640, 12320, 64, 16), (700, 12544, 192, 8), (1100, 7456, 128, 40), (768, 12288, 64, 128),
                                        (16400, 768, 64, 16), (4100, 96, 96, 8), (5000, 320, 32, 24)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tiles(T, N, K, rank, dtype):
    g = torch.Generator().manual_seed(T)
    cuts = torch.sort(torch.randint(T, (6,), generator=g))[0].tolist() + [T]
    index, at = [], 0
    for a, c in zip([2, -1, 0, 2, 4, 1, 0], cuts):  # runs, an adapter that comes back, one (3) without tokens
        index += [a] * (c - at)
        at = c
    c = case(T, N, K, 5, rank, dtype, index, bs=32 if K % 64 else 64, dq=True)
    bias = torch.randn(N, generator=g).to(dtype).cuda()
    check_forward(c, forward(c, bias=bias), bias)
    check_forward(c, forward(c, out_dtype=torch.float32))
    c = case(T, K, N, 5, rank, dtype, index, bs=32, dq=True)  # backward: its outputs are K wide
    check_backward(c, backward(c))


@pytest.mark.parametrize("T", [700, 1000])
def test_tiles_of_many_adapters(T):
    """Every row of a tile with another adapter, in no order."""
    g = torch.Generator().manual_seed(3)
    c = case(T, 12320, 64, 90, 16, BF, torch.randint(-1, 90, (T,), generator=g))
    check_forward(c, forward(c))
    c = case(T, 64, 12320, 90, 16, BF, torch.randint(-1, 90, (T,), generator=g), bs=32)
    check_backward(c, backward(c))


def sorted_parts(T, parts):
    out = []
    for a, n in parts:
        out += [a] * n
    assert len(out) == T
    return out


INDEX = {
    "none": [-1] * 600, "one": [0] * 600, "outside": [5, -7, 2 ** 31 - 1, -2 ** 31] * 150, "turns": [0, 1, 2, 3, 4] * 120,
    "parts": sorted_parts(600, [(2, 255), (0, 1), (-1, 2), (4, 300), (1, 42)]), "last": [-1] * 599 + [4], "unused": [1, 3] * 300,
    "falling": sorted_parts(600, [(4, 130), (3, 126), (2, 129), (1, 127), (0, 88)]),
}


@pytest.mark.parametrize("kind", sorted(INDEX))
@pytest.mark.parametrize("T", [12, 600])
def test_index(kind, T):
    c = case(T, 320, 256, 5, 32, BF, INDEX[kind][:T])
    check_forward(c, forward(c))
    grads = backward(c)
    check_backward(c, grads)
    for a in range(5):
        if a not in INDEX[kind][:T]:
            assert (grads[1][a] == 0).all() and (grads[2][a] == 0).all()


def test_many_adapters():
    c = case(500, 64, 64, 300, 8, BF)
    check_forward(c, forward(c))
    check_backward(c, backward(c))


def test_without_adapters_it_is_the_product():
    for T in (1, 30, 300):
        c = case(T, 256, 512, 2, 16, BF, [-1] * T)
        f = qmv.gemv_4bit if T <= 8 else qmv.gemm_4bit
        R.check_lora(f(c["x"], c["packed"], c["state"]), c["x"], c["W"], c["down"], c["up"], c["scale"], c["index"])
        check_forward(c, forward(c))


def test_adapter_alone_is_precise():
    """A projection of zeros: what is left is the adapter's part, whose inner
    values must not have been rounded to one 16-bit number."""
    for dtype in (BF, HF):
        for T in (5, 300, 600):
            c = case(T, 256, 512, 3, 32, dtype)
            c["packed"].fill_(0x77)
            c["W"] = torch.zeros_like(c["W"])
            check_forward(c, forward(c, out_dtype=torch.float32))


def test_gradients_against_differences():
    """f(w + h) - f(w - h) of f = sum(dy y) against the gradient along 2h.  y is
    linear in each operand, so nothing is left but roundings: those of y's sums
    on one side, those of the gradients on the other (the weights' own to fp16
    are the same on both, up to one rounding of a product by the block scale)."""
    T, N, K, n, rank = 70, 96, 128, 3, 8
    c = case(T, N, K, n, rank, HF)
    grads = dict(zip(("x", "down", "up"), (t.double().cpu() for t in backward(c, grad_dtype=torch.float32))))
    x, dy, W, down, up, scale = (c[k].double().cpu() for k in ("x", "dy", "W", "down", "up", "scale"))
    i = c["index"].cpu()
    s = torch.where(i >= 0, scale[i.clamp(min=0).long()], 0.0)
    D, B = down[i.clamp(min=0).long()], up[i.clamp(min=0).long()]          # [T, R, K], [T, N, R]
    mx, mdy, mW, mD, mB = x.abs() + 0.25, dy.abs(), W.abs(), D.abs() + 0.25, B.abs() + 0.25
    inner = s[:, None] * torch.einsum("tk,trk->tr", mx, mD)
    base, part = mx @ mW.T, torch.einsum("tr,tnr->tn", inner, mB)
    u = R.U[HF]
    err_y = 2 * (mdy * (R.c32(K) * base + (u * u + 2 * R.c32(K)) * part + 2.0 ** -25 * mB.sum(2))).sum().item()
    back = s[:, None] * torch.einsum("tn,tnr->tr", mdy, mB)
    mags = {"x": (mdy @ mW + torch.einsum("tr,trk->tk", back, mD)).sum() * (u + u + R.c32(N)),
            "down": torch.einsum("tr,tk->rk", back, mx).sum() * (u * u + 2 * R.c32(N + T)) + 2.0 ** -25 * mx.sum() * rank,
            "up": torch.einsum("tn,tr->nr", mdy, inner).sum() * (u * u + 2 * R.c32(K + T)) + 2.0 ** -25 * mdy.sum() * rank}
    g = torch.Generator().manual_seed(9)
    for name, grad in grads.items():
        h = ((torch.randint(0, 2, c[name].shape, generator=g) * 2 - 1) * 0.25).to(HF).cuda()
        f, at = [], []
        for sign in (1, -1):
            args = {k: c[k] for k in ("x", "down", "up")}
            args[name] = (args[name] + sign * h).contiguous()
            at.append(args[name].double().cpu())
            y = qmv.lora_4bit(args["x"], c["packed"], c["state"], qmv.LoraAdapters(args["down"], args["up"], c["scale"]),
                              c["index"], out_dtype=torch.float32)
            f.append((dy * y.double().cpu()).sum().item())
        want = (grad * (at[0] - at[1])).sum().item()
        assert abs(f[0] - f[1] - want) <= 1.01 * (err_y + 0.51 * mags[name].item()), name


def test_strided_and_batched_rows():
    c = case(48, 128, 256, 3, 16, BF)
    wide = torch.zeros(48, 2, 256, dtype=BF, device="cuda")
    wide[:, 1] = c["x"]
    ref = forward(c)
    assert torch.equal(qmv.lora_4bit(wide[:, 1], c["packed"], c["state"], c["adapters"], c["index"]), ref)
    three = c["x"].view(6, 8, 256)
    assert torch.equal(qmv.lora_4bit(three, c["packed"], c["state"], c["adapters"], c["index"].view(6, 8)), ref)
    every = torch.stack([c["index"]] * 2, 1)[:, 0]  # strided numbers
    assert torch.equal(qmv.lora_4bit(c["x"], c["packed"], c["state"], c["adapters"], every), ref)
    out = torch.empty(48, 128, dtype=BF, device="cuda")
    assert forward(c, out=out) is out and torch.equal(out, ref)


def test_no_tokens():
    c = case(4, 64, 64, 2, 8, BF)
    x, i = c["x"][:0], c["index"][:0]
    assert qmv.lora_4bit(x, c["packed"], c["state"], c["adapters"], i).shape == (0, 64)
    dx, dd, du = qmv.lora_4bit_backward(c["dy"][:0], x, c["packed"], c["state"], c["adapters"], i)
    assert dx.shape == (0, 64) and (dd == 0).all() and (du == 0).all()


def test_a_row_that_is_not_finite_stays_alone():
    for T, N, K in ((5, 128, 256), (40, 128, 256), (600, 128, 256), (700, 12320, 64)):
        c = case(T, N, K, 3, 16, BF)
        ref = forward(c)
        x = c["x"].clone()
        x[1, 3], x[T - 2, 50] = float("nan"), float("inf")
        y = qmv.lora_4bit(x, c["packed"], c["state"], c["adapters"], c["index"])
        rest = [t for t in range(T) if t not in (1, T - 2)]
        assert torch.equal(y[rest], ref[rest]) and not torch.isfinite(y[1]).any()


def test_widest_backward():
    """More columns than 256 rows of fp32 sums have room for in 2^31 bytes; the last of them."""
    T, N, K, rank, last = 300, 32, (1 << 21) + 288, 8, 320
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    packed, state = qmv.quantize_4bit(rnd(N, K), 32, "nf4")
    dy, x, down, up = rnd(T, N), rnd(T, K), rnd(2, rank, K), rnd(2, N, rank)
    index = (torch.arange(T, device="cuda") % 3 - 1).int()
    scale = torch.ones(2, device="cuda")
    dx, _, _ = qmv.lora_4bit_backward(dy, x, packed, state, qmv.LoraAdapters(down, up, scale), index)
    W = qmv.dequantize_4bit(packed, state, out_dtype=torch.float32)
    for cut in (slice(0, last), slice(K - last, K)):  # the forward's formula, with the two factors in each other's place
        R.check_lora(dx[:, cut], dy, W[:, cut].T, up.transpose(1, 2), down[..., cut].transpose(1, 2), scale, index, what="dx")


@pytest.mark.parametrize("T,N,K", [(6, 192, 320), (90, 192, 320), (300, 192, 320), (700, 12320, 64)])
def test_an_adapter_that_is_not_finite_spoils_its_own_tokens_only(T, N, K):
    """Its tokens share tiles with others' and with tokens that have no adapter."""
    g = torch.Generator().manual_seed(T)
    index = torch.randint(-1, 3, (T,), generator=g)
    index[:3] = torch.tensor([0, 1, -1])
    others = (index != 1).cuda()

    def spoil(c):
        down, up = c["down"].clone(), c["up"].clone()
        down[1, 3, 5], up[1, 7, 2], up[1, 9, 4] = float("inf"), float("inf"), float("nan")
        return dict(c, down=down, up=up, adapters=qmv.LoraAdapters(down, up, c["scale"]))

    c = case(T, N, K, 3, 16, BF, index)
    assert torch.equal(forward(spoil(c))[others], forward(c)[others])
    c = case(T, K, N, 3, 16, BF, index, bs=32)
    want, got = backward(c), backward(spoil(c))
    assert torch.equal(got[0][others], want[0][others])
    for a in (0, 2):
        assert torch.equal(got[1][a], want[1][a]) and torch.equal(got[2][a], want[2][a])


@pytest.mark.parametrize("T,N,K", [(5, 192, 320), (90, 192, 320), (600, 192, 320), (700, 12320, 64)])
def test_repeats_and_graphs(T, N, K):
    """The same bits every time, in a captured graph too, whose replays follow
    new inputs, with eager calls of other sizes between them."""
    c, other = case(T, N, K, 4, 16, BF), case(T + 70, N, K, 4, 16, BF)
    y, grads = forward(c), backward(c)
    assert torch.equal(forward(c), y) and all(torch.equal(a, b) for a, b in zip(backward(c), grads))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        forward(c), backward(c)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, ggrads = forward(c), backward(c)
    x0 = c["x"].clone()
    for i in range(3):
        c["x"].copy_(x0 if i != 1 else -x0)
        graph.replay()
        forward(other), backward(other)
        torch.cuda.synchronize()
        want_y, want = forward(c), backward(c)
        assert torch.equal(gy, want_y) and all(torch.equal(a, b) for a, b in zip(ggrads, want))


def test_two_streams():
    """Calls on two streams at once have workspaces of their own."""
    a, b = case(300, 256, 512, 3, 16, BF), case(300, 256, 512, 3, 16, BF, seed=5)
    ya, yb = forward(a), forward(b)
    ga, gb = backward(a), backward(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, (s, c) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i].append((forward(c), *backward(c)))
    torch.cuda.synchronize()
    for i, want in enumerate(((ya, *ga), (yb, *gb))):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want))
