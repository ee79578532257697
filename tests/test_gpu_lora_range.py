"""Adapters' inner values u = scale down x and v = scale up^T dy over fp16's whole
range and beyond: small ones as where a training starts (up near zero, small
dy), ones above 65504, and tokens that differ by powers of two.

Bounds, beside those of tuning_reference: a token's inner values are two 16-bit
terms times a power of two that brings the largest of them to 2^14 or more (where it is
within 2^-64 .. 2^92).  The second term is off by half of fp16's smallest number at most,
2^-25, so a value is off by 2^-22 of itself or 2^-39 of its token's largest; taken as 2^-38,
since the largest is known up to its own sums' roundings.  In the adapters' gradients all tokens of a run are
brought to the power of two of the run's largest: that rounds both terms once
more, 2^-25 each, or drops what is below 2^-24 in all, so a value is off by
3 x 2^-25 / 2^14 < 2^-37 of the largest of its adapter, taken as 2^-36."""
import pytest
import torch

import quantized_matvec_amd as qmv
import tuning_reference as R

pytestmark = pytest.mark.gpu
HF, F32 = torch.float16, torch.float32
T2 = 2.0 ** -22


def zero_weight(N, K, bs=32):
    """A projection of zeros: what is left is the adapters' part."""
    packed = torch.full((N * K // 2,), 0x77, dtype=torch.uint8, device="cuda")
    return packed, qmv.QuantState((N, K), HF, bs, "nf4", absmax=torch.ones(N * K // bs, device="cuda"))


def case(T, N, K, n=3, rank=16, x=1.0, dy=1.0, down=1.0, up=1.0, scale=1.0, spread=0, seed=1):
    """Normal values times x, dy, down and up; each token's rows of x and dy times a power of two in 2^-spread .. 1."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda gain, *s: torch.randn(*s, generator=g) * gain
    each = 2.0 ** -torch.randint(0, spread + 1, (T, 1), generator=g).float()
    each[T // 2] = 1.0
    index = torch.randint(-1, n, (T,), generator=g).sort()[0].int()
    down, up = rnd(down, n, rank, K).to(HF).cuda(), rnd(up, n, N, rank).to(HF).cuda()
    scale = (scale * (0.5 + torch.rand(n, generator=g))).cuda()
    return dict(x=(rnd(x, T, K) * each).to(HF).cuda(), dy=(rnd(dy, T, N) * each).to(HF).cuda(), w=zero_weight(N, K), down=down, up=up,
                scale=scale, index=index.cuda(), adapters=qmv.LoraAdapters(down, up, scale))


def largest(v):
    return v.abs().amax() if len(v) else torch.zeros(())


def check(c, forward=True):
    x, dy, down, up, scale = (c[k].double().cpu() for k in ("x", "dy", "down", "up", "scale"))
    (T, K), N, R2 = x.shape, dy.shape[1], 2 * down.shape[1]
    index = c["index"].cpu()
    y = qmv.lora_4bit(c["x"], *c["w"], c["adapters"], c["index"], out_dtype=F32) if forward else None
    dx, dd, du = qmv.lora_4bit_backward(c["dy"], c["x"], *c["w"], c["adapters"], c["index"], grad_dtype=F32)
    ry, by = torch.zeros(T, N).double(), torch.zeros(T, N).double()
    rx, bx = torch.zeros(T, K).double(), torch.zeros(T, K).double()
    for a in range(len(down)):
        t = (index == a).nonzero()[:, 0]
        s = scale[a].abs()
        u, mu = scale[a] * (x[t] @ down[a].T), s * (x[t].abs() @ down[a].abs().T)
        v, mv = scale[a] * (dy[t] @ up[a]), s * (dy[t].abs() @ up[a].abs())
        top = lambda w: 2.0 ** -38 * w.abs().amax(1, keepdim=True)
        ry[t], by[t] = u @ up[a].T, (T2 + R.c32(K) + R.c32(R2)) * (mu @ up[a].abs().T) + top(u) * up[a].abs().sum(1)
        rx[t], bx[t] = v @ down[a], (T2 + R.c32(N) + R.c32(R2)) * (mv @ down[a].abs()) + top(v) * down[a].abs().sum(0)
        b = (T2 + R.c32(N) + R.c32(2 * T)) * (mv.T @ x[t].abs()) + 2.0 ** -36 * largest(v) * x[t].abs().sum(0)
        r = v.T @ x[t]
        R._check(dd[a], r, R._rounded(r, b, F32), f"d_down[{a}]")
        b = (T2 + R.c32(K) + R.c32(2 * T)) * (dy[t].abs().T @ mu) + 2.0 ** -36 * largest(u) * dy[t].abs().sum(0)[:, None]
        r = dy[t].T @ u
        R._check(du[a], r, R._rounded(r, b, F32), f"d_up[{a}]")
    if forward:
        R._check(y, ry, R._rounded(ry, by, F32), "y")
    R._check(dx, rx, R._rounded(rx, bx, HF), "dx")


# what x, dy, down, up and scale are like; dx has to lie in fp16's range to show anything
KINDS = {
    "training starts": dict(dy=1e-4, up=1e-4, down=8.0),
    "smallest": dict(x=2.0 ** -12, dy=2.0 ** -16, down=2.0 ** -3, up=2.0 ** -17, scale=2.0 ** -10),
    "above 65504": dict(x=60.0, dy=60.0, down=8.0, up=8.0, scale=500.0),  # dx: see below
    "uneven": dict(spread=14, down=0.25, up=0.25),
    "uneven and small": dict(spread=14, down=4.0, up=2.0 ** -12, dy=2.0 ** -4),
}


@pytest.mark.parametrize("kind", sorted(KINDS))
# tokens before and after the rules that choose a kernel; the last two by the tile product, forward and backward
@pytest.mark.parametrize("T,N,K", [(20, 96, 128), (64, 96, 128), (65, 96, 128), (300, 352, 320), (700, 352, 320), (700, 12320, 64), (700, 64, 12320)])
def test_ranges(T, N, K, kind):
    c = case(T, N, K, **KINDS[kind])
    if kind == "above 65504":  # down of 2^-6 in every fourth column only, so that dx is finite while u is not small
        c["down"].mul_((torch.arange(K, device="cuda") % 4 == 0).to(HF)).clamp_(-2.0 ** -6, 2.0 ** -6)
        c["x"].mul_(256).clamp_(-32768, 32768)
        c["dy"].clamp_(-8, 8)
        c["up"].clamp_(-0.25, 0.25)
        c["up"].mul_(0.125)
        c["scale"].fill_(40.0)
    check(c)


@pytest.mark.parametrize("rank", [8, 24, 64, 128])
@pytest.mark.parametrize("T,N,K", [(300, 96, 128), (660, 64, 12320)])
def test_ranks(T, N, K, rank):
    check(case(T, N, K, rank=rank, dy=1e-4, up=1e-4, down=8.0, spread=6))


def test_runs_of_many_windows():
    """One adapter over several windows of the gradients, each with a power of two of its own."""
    c = case(2100, 64, 96, n=1, rank=16, dy=1e-3, up=1e-3, down=2.0)
    for i, f in enumerate((1.0, 2.0 ** -12, 1.0, 0.0, 2.0 ** -8, 1.0)):
        c["x"][350 * i:350 * (i + 1)] *= f
        c["dy"][350 * i:350 * (i + 1)] *= f
    check(c)


@pytest.mark.parametrize("T,N,K", [(90, 96, 128), (700, 12320, 64)])
def test_a_token_depends_on_no_other(T, N, K):
    """A token's bits are the same beside a token of its adapter that is 2^13 times as large, or not finite."""
    c = case(T, N, K, n=1, x=2.0 ** -6, dy=2.0 ** -6, up=2.0 ** -12)
    y = qmv.lora_4bit(c["x"], *c["w"], c["adapters"], c["index"], out_dtype=F32)
    rest = [t for t in range(T) if t != T - 2]
    for f in (2.0 ** 13, float("inf"), float("nan")):
        x = c["x"].clone()
        x[T - 2] *= f
        assert torch.equal(qmv.lora_4bit(x, *c["w"], c["adapters"], c["index"], out_dtype=F32)[rest], y[rest])
    # the backward's outputs are K wide
    c = case(T, K if K % 32 == 0 else 32, N, n=1, x=2.0 ** -6, dy=2.0 ** -6, up=2.0 ** -12, down=64.0)
    dx = qmv.lora_4bit_backward(c["dy"], c["x"], *c["w"], c["adapters"], c["index"])[0]
    for f in (2.0 ** 13, float("inf"), float("nan")):
        dy = c["dy"].clone()
        dy[T - 2] *= f
        assert torch.equal(qmv.lora_4bit_backward(dy, c["x"], *c["w"], c["adapters"], c["index"])[0][rest], dx[rest])


def test_tokens_without_an_adapter_and_zeros_beside_the_projection():
    """Rows of zeros in an adapter, and rows of none, keep the projection's bits beside those of others."""
    T, N, K = 700, 12320, 64
    g = torch.Generator().manual_seed(4)
    packed, state = qmv.quantize_4bit((torch.randn(N, K, generator=g) * 0.125).to(HF).cuda(), 64, "nf4")
    x = torch.randn(T, K, generator=g).to(HF).cuda()
    down, up = torch.randn(2, 16, K, generator=g).to(HF).cuda(), torch.randn(2, N, 16, generator=g).to(HF).cuda()
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    some = (torch.arange(T, device="cuda") % 3 - 1).int()
    down[1] = 0
    adapters = qmv.LoraAdapters(down, up, 1.0)
    for out in (HF, F32):
        y = qmv.lora_4bit(x, packed, state, adapters, some, out_dtype=out)
        plain = qmv.lora_4bit(x, packed, state, adapters, none, out_dtype=out)
        assert torch.equal(y[some != 0], plain[some != 0]) and not torch.equal(y, plain)
