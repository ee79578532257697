"""lora_4bit, its backward and the losses at the sizes of large models' calls with few
tokens, where work is divided in ways that smaller sizes do not come to: several turns
of columns and several slices of the sum (17 to 64 tokens), the backward that divides its
sum among workgroups, and vocabularies in several pieces.  Each test says which.
Against float64, with the bounds of tuning_reference."""
import pytest
import torch

import quantized_matvec_amd as qmv
import tuning_reference as R
from test_gpu_lora import backward, case, check_backward, check_forward, forward
from test_gpu_loss import both, dlosses, rows, targets, teacher, weight, whole_weight

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


# 17 to 64 tokens: slices of 512 terms, and workgroups that each go over columns in turns of 256: with 8 slices 8192
# columns a turn (one turn and a part; two and a part, the last not whole), with 9 slices, the last of 64 terms, 7168;
# with 15 slices 4352
@pytest.mark.parametrize("N,K", [(9000, 4096), (16500, 4096), (8000, 4160), (4400, 7680)])
@pytest.mark.parametrize("T", [17, 32, 33, 50, 64])
@pytest.mark.parametrize("dtype,dq", [(BF, True), (HF, False)])
def test_adapters_of_a_decode_step(T, N, K, dtype, dq):
    c = case(T, N, K, 3, 16, dtype, dq=dq)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    check_forward(c, forward(c, bias=bias), bias)
    check_forward(c, forward(c, out_dtype=F32))


# the same product's logits, whose slices are added up; the gradient by gemm_4bit_backward's kernel that divides the
# sum among workgroups (K a multiple of 256, enough weights for it), but for 320 (the tile product)
@pytest.mark.parametrize("V,K", [(9001, 4096), (16500, 4096), (33000, 320)])
@pytest.mark.parametrize("T", [17, 33, 64])
@pytest.mark.parametrize("dtype,dq", [(BF, True), (HF, False)])
def test_losses_of_few_tokens(T, V, K, dtype, dq):
    w = weight(V, K, dq=dq, dtype=dtype)
    both(rows(T, K, dtype), w, targets(T, V), dlosses(T))


# that backward, and the last V % 64 columns, which it leaves to the last kernel: none, one, 37, 63
@pytest.mark.parametrize("V", [4160, 4161, 4133, 4159])
@pytest.mark.parametrize("T", [1, 5, 40, 200, 447])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_divided_backward_and_last_columns(T, V, dtype):
    K = 4096
    w = weight(V, K, dtype=dtype)
    x, t = rows(T, K, dtype), targets(T, V)
    t[0] = V - 1  # a target among the last columns
    both(x, w, t, dlosses(T))


@pytest.mark.parametrize("T", [5, 200])
def test_divided_backward_of_a_divergence(T):
    V, K = 4133, 4096
    packed, state, W = weight(V, K, dq=True)
    x, g = rows(T, K, BF), dlosses(T)
    ids, z = teacher(T, V, 9, F32)
    ids[:, 3] = V - 2
    loss, dx = qmv.distill_4bit(x, packed, state, ids, z, 2.0, g, loss_dtype=F32)
    R.check_loss(loss, dx, x, W, ids, z, 2.0, g)


# 447 tokens: pieces of 147456 columns, 64 tokens with 16 slices: of 65536; the second's sums are added to
# the first's, rescaled.  The second's last columns are 4 and 16.
@pytest.mark.parametrize("T,V,K", [(447, 147456 + 4100, 512), (64, 65536 + 464, 8192)])
@pytest.mark.parametrize("grows", [False, True])
def test_divided_backward_in_pieces(T, V, K, grows):
    first = 147456 if T == 447 else 65536
    packed, state, W = weight(V, K)
    # the second piece's logits reach further up than the first's, or less far
    state.absmax.view(V, -1).mul_(torch.where(torch.arange(V) < first, 0.5 if grows else 1.0, 1.0 if grows else 0.5)[:, None].cuda())
    W = qmv.dequantize_4bit(packed, state, out_dtype=F32)
    t = targets(T, V)
    t[0], t[1], t[2], t[3] = first - 1, first, V - 1, V
    both(rows(T, K, BF), (packed, state, W), t, dlosses(T))


def moved(V, K, border, low, high):
    """Exact weights whose rows from `border` on are `high` times as large, the others `low` times."""
    packed, state, _ = whole_weight(V, K)
    state.absmax.view(V, 1).mul_(torch.where(torch.arange(V) < border, low, high)[:, None].cuda())
    return packed, state, qmv.dequantize_4bit(packed, state, out_dtype=F32)


# Pieces of 32768 columns up to 1792 tokens, of 16384 from there on; the tile product from 448 tokens, below it for the
# gradient's part only.  Logits in the thousands in one piece, and in the tens in the other: the maximum moves
# from piece to piece, and what has been added up is rescaled, or stays and outweighs the rest.
@pytest.mark.parametrize("T,V", [(4, 33500), (40, 33500), (300, 33500), (500, 33500), (500, 66000), (1800, 20000), (1800, 33000)])
@pytest.mark.parametrize("low,high", [(1.0, 64.0), (64.0, 1.0), (1.0, 1.25)])
def test_a_maximum_that_moves_from_piece_to_piece(T, V, low, high):
    K = 64
    x = rows(T, K, BF, whole=True) * 8
    border = 16384 if V <= 20000 else 32768
    w = moved(V, K, border, low, high)
    t = targets(T, V)
    t[0], t[1], t[2] = border - 1, border, V - 1
    both(x, w, t, dlosses(T), whole=(low, high) != (1.0, 1.25))


# the input's gradient by the kernel that divides its sum among workgroups
@pytest.mark.parametrize("T", [1, 40, 129, 500])
@pytest.mark.parametrize("dtype,dq", [(BF, True), (HF, False)])
def test_adapters_backward_by_the_divided_kernel(T, dtype, dq):
    c = case(T, 4160, 4096, 3, 16, dtype, dq=dq)
    check_backward(c, backward(c))


def test_gradients_along_their_signs():
    """f(w + h) - f(w - h) of f = sum(dy y) against the gradient along 2h, for h along the
    signs of the exact gradient and of the adapters' part of it, so that what is compared is a sum of magnitudes:
    a gradient of zeros, or one without that part, is far off.  y is linear in each operand.  Off are y's sums on
    one side (tuning_reference's bounds without the weights' rounding, which is the same in both), the gradient's
    sums and rounding on the other."""
    T, N, K, n, rank = 70, 96, 128, 3, 8
    c = case(T, N, K, n, rank, HF)
    got = dict(zip(("x", "down", "up"), (t.double().cpu() for t in backward(c, grad_dtype=F32))))
    x, dy, W, down, up, scale = (c[k].double().cpu() for k in ("x", "dy", "W", "down", "up", "scale"))
    i = c["index"].cpu()
    s = torch.where(i >= 0, scale[i.clamp(min=0).long()], 0.0)[:, None]
    at = i.clamp(min=0).long()
    bm = lambda a, b: (a[:, None, :] * b).sum(2)  # [T, j] with [T, i, j]
    u, v = s * bm(x, down[at]), s * bm(dy, up[at].transpose(1, 2))
    mine = [(i == a).nonzero()[:, 0] for a in range(n)]
    parts = {"x": (dy @ W, bm(v, down[at].transpose(1, 2))),
             "down": (0.0, torch.stack([v[t].T @ x[t] for t in mine])), "up": (0.0, torch.stack([dy[t].T @ u[t] for t in mine]))}
    U = R.U[HF]
    for name, (base, adapter) in parts.items():
        exact = base + adapter
        for along in (exact, adapter):
            h = (along.sign() * 0.25).to(HF).cuda()
            f, moved_to, err = [], [], 0.0
            for sign in (1, -1):
                args = {k: c[k] for k in ("x", "down", "up")}
                args[name] = (args[name] + sign * h).contiguous()
                moved_to.append(args[name].double().cpu())
                y = qmv.lora_4bit(args["x"], c["packed"], c["state"], qmv.LoraAdapters(args["down"], args["up"], c["scale"]),
                                  c["index"], out_dtype=F32)
                f.append((dy * y.double().cpu()).sum().item())
                X, D, B = (args[k].double().cpu().abs() for k in ("x", "down", "up"))
                inner = s * bm(X, D[at])
                my = R.c32(K) * (X @ W.abs().T) + (U * U + R.c32(K) + R.c32(2 * rank)) * bm(inner, B[at])
                err += (dy.abs() * (my + 2.0 ** -38 * inner.amax(1, keepdim=True) * B[at].sum(2))).sum().item()
            step = moved_to[0] - moved_to[1]
            mv, mu = s * bm(dy.abs(), up[at].abs().transpose(1, 2)), s * bm(x.abs(), down[at].abs())
            mag = {"x": lambda: (U + R.c32(N)) * (dy.abs() @ W.abs()) + (U + U * U + R.c32(N) + R.c32(2 * rank)) * bm(mv, down[at].abs().transpose(1, 2)),
                   "down": lambda: (U * U + R.c32(N) + R.c32(2 * T)) * torch.stack([mv[t].T @ x[t].abs() for t in mine]) + 2.0 ** -36 * mv.max() * x.abs().sum(0),
                   "up": lambda: (U * U + R.c32(K) + R.c32(2 * T)) * torch.stack([dy[t].abs().T @ mu[t] for t in mine]) + 2.0 ** -36 * mu.max() * dy.abs().sum(0)[:, None]}[name]()
            err += (mag * step.abs()).sum().item()
            want, size = (exact * step).sum().item(), (adapter.abs() * step.abs()).sum().item()
            # the weights' rounding: the exact values are of the unrounded ones
            err_w = U * ((dy.abs() @ W.abs()) * step.abs()).sum().item() if name == "x" else 0.0
            assert err + err_w < 0.05 * size, name  # the bound itself: a twentieth of the part that has to be seen
            assert abs(f[0] - f[1] - (got[name] * step).sum().item()) <= 1.01 * err, name
            assert abs(f[0] - f[1] - want) <= 1.01 * (err + err_w), name
