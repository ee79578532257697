"""examples/finetune_4bit.py: it runs, repeats, and its gradients are those of the
same model written with torch in float64 over the dequantized weights."""
import importlib.util
import os

import pytest
import torch

import quantized_matvec_amd as qmv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("finetune_4bit", os.path.join(ROOT, "examples", "finetune_4bit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model, tokens, index, loss_of):
    """Loss and gradients of the adapters in float64 on the CPU."""
    w = lambda pair: qmv.dequantize_4bit(*pair, out_dtype=torch.float32).double().cpu()
    params = [p.detach().double().cpu().requires_grad_() for p in model.parameters()]
    index = index.long().cpu()
    on = (index >= 0)[:, None]
    scale = model.scale.double().cpu()[index.clamp(min=0)][:, None]

    def lora(x, weight, down, up):
        u = torch.einsum("tk,trk->tr", x, down[index.clamp(min=0)]) * scale * on
        return x @ w(weight).T + torch.einsum("tr,tnr->tn", u, up[index.clamp(min=0)])
    norm = lambda x: torch.nn.functional.rms_norm(x, x.shape[-1:])
    x = w(model.embedding)[tokens.cpu()] * 16
    for i, (w_in, w_out) in enumerate(model.layers):
        y = lora(norm(x), w_in, *params[4 * i:4 * i + 2])
        x = x + lora(torch.nn.functional.silu(y), w_out, *params[4 * i + 2:4 * i + 4])
    loss = loss_of(norm(x) @ w(model.head).T)
    loss.backward()
    return loss.item(), [p.grad for p in params]


def check(model, loss, gain, want, dtype):
    """Along the way from an adapter to the loss and back there are, for two
    layers, fewer than 32 roundings to 16 bits (the rows of each operator, its
    weights, the two norms' and the activation's outputs, and as many backward), each of half a step.
    Norms and silu stretch a relative error by no more than 2 here, so with
    independent roundings sqrt(32) * 2 of them, and 4 times that for all."""
    ref, grads = want
    tol = 4 * 2 * 32 ** 0.5 * U[dtype]
    assert abs(loss.item() / gain - ref) <= tol * abs(ref)
    loss.backward()
    for p, g in zip(model.parameters(), grads):
        off = (p.grad.double().cpu() / gain - g).norm()
        assert torch.isfinite(p.grad).all() and off <= tol * g.norm(), (off / g.norm()).item()


@pytest.mark.parametrize("dtype,gain", [(torch.bfloat16, 1.0), (torch.float16, 256.0)])
@pytest.mark.parametrize("lengths", [[40, 33, 70, 9], [700, 1, 2, 300]])
def test_gradients(example, dtype, gain, lengths):
    model = example.Model(dtype=dtype)
    tokens, index, target = example.batch(lengths, 512, [min(n, 4) for n in lengths])
    index[-5:] = -1
    t = target.cpu()
    want = reference(model, tokens, index, lambda l: torch.nn.functional.cross_entropy(l, t, ignore_index=-100))
    check(model, model.loss(tokens, index, target, gain), gain, want, dtype)
    first = [p.grad.clone() for p in model.parameters()]
    for p in model.parameters():
        p.grad = None
    model.loss(tokens, index, target, gain).backward()
    assert all(torch.equal(a, p.grad) for a, p in zip(first, model.parameters()))


@pytest.mark.parametrize("dtype,gain", [(torch.bfloat16, 1.0), (torch.float16, 256.0)])
def test_distillation_gradients(example, dtype, gain):
    model = example.Model(dtype=dtype)
    tokens, index, _ = example.batch([40, 33, 70, 9], 512, [0] * 4)
    g = torch.Generator().manual_seed(1)
    ids = torch.stack([torch.randperm(512, generator=g)[:8] for _ in range(len(tokens))])
    teacher = torch.randn(len(tokens), 8, generator=g)

    def loss_of(l):
        p = (teacher.double() / 2).softmax(-1)
        logq = (l / 2).log_softmax(-1).gather(1, ids)
        return (p * (p.log() - logq)).sum(-1).mean()
    want = reference(model, tokens, index, loss_of)
    check(model, model.distill(tokens, index, ids.cuda(), teacher.cuda(), 2.0, gain), gain, want, dtype)


def test_runs(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["finetune_4bit.py", "2"])
    example.main()
    out = capsys.readouterr().out
    assert out.count("loss") == 2 and "teacher" in out and "nan" not in out
