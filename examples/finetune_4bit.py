"""Fine-tuning low-rank adapters beside frozen 4-bit weights, for two tasks at once.

Random weights: embedding_4bit -> residual blocks whose two
projections are lora_4bit -> cross_entropy_4bit over a 4-bit vocabulary.  A
batch packs the sequences of both tasks, each token with its task's adapter
(index), prompts do not count (target -100), and torch's autograd carries the
gradients between the library's calls.  At the end the second task is also
pulled towards a teacher's largest logits (distill_4bit).

    python examples/finetune_4bit.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matvec_amd as qmv  # noqa: E402
from quantized_matvec_amd.qmv import embedding_4bit  # noqa: E402


class LoraLinear(torch.autograd.Function):
    """y = W_hat x + the token's adapter, with the gradients of x and of the adapters."""

    @staticmethod
    def forward(ctx, x, down, up, scale, weight, index):
        ctx.save_for_backward(x, down, up)
        ctx.rest = scale, weight, index
        return qmv.lora_4bit(x, *weight, qmv.LoraAdapters(down, up, scale), index)

    @staticmethod
    def backward(ctx, dy):
        x, down, up = ctx.saved_tensors
        scale, weight, index = ctx.rest
        dx, d_down, d_up = qmv.lora_4bit_backward(dy, x, *weight, qmv.LoraAdapters(down, up, scale), index)
        return dx, d_down, d_up, None, None, None


class MeanLoss(torch.autograd.Function):
    """The mean of a loss over the tokens that count; its gradient comes with it."""

    @staticmethod
    def forward(ctx, x, call, count, gain):
        # gain: a loss scale, so that gradients of few parts of a thousand do not fall under fp16's smallest numbers
        loss, ctx.dx = call(x, torch.full((x.shape[0],), gain / max(count, 1), dtype=torch.float32, device=x.device))
        return gain * loss.sum() / max(count, 1)

    @staticmethod
    def backward(ctx, d):
        return (ctx.dx.float() * d).to(ctx.dx.dtype), None, None, None


class Model:
    def __init__(self, vocab=512, width=256, mlp=512, layers=2, tasks=2, rank=8, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)
        weight = lambda n, k: qmv.quantize_4bit((rnd(n, k) * k ** -0.5).to(dtype), 64, "nf4", double_quant=True)
        self.dtype, self.device = dtype, device
        self.scale = torch.full((tasks,), 2.0, device=device)
        self.embedding, self.head = weight(vocab, width), weight(vocab, width)
        self.layers = [(weight(mlp, width), weight(width, mlp)) for _ in range(layers)]
        # up starts near zero, so that training starts from the frozen model's outputs
        self.adapters = [[((rnd(tasks, rank, k) * k ** -0.5).to(dtype).requires_grad_(), (rnd(tasks, n, rank) * 0.02).to(dtype).requires_grad_())
                          for n, k in ((mlp, width), (width, mlp))] for _ in range(layers)]

    def parameters(self):
        return [p for layer in self.adapters for pair in layer for p in pair]

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)

    def hidden(self, tokens, index):
        x = embedding_4bit(tokens, *self.embedding, out_dtype=self.dtype)
        x = (x.float() * 16).to(self.dtype)  # rows of unit size
        for (w_in, w_out), (a_in, a_out) in zip(self.layers, self.adapters):
            y = LoraLinear.apply(self.norm(x), *a_in, self.scale, w_in, index)
            x = x + LoraLinear.apply(torch.nn.functional.silu(y), *a_out, self.scale, w_out, index)
        return self.norm(x)

    def loss(self, tokens, index, target, gain=1.0):
        count = int((target >= 0).sum())  # the program's own batch: known without the GPU
        call = lambda x, d: qmv.cross_entropy_4bit(x, *self.head, target, d, loss_dtype=torch.float32)
        return MeanLoss.apply(self.hidden(tokens, index), call, count, gain)

    def distill(self, tokens, index, ids, teacher, temperature=2.0, gain=1.0):
        call = lambda x, d: qmv.distill_4bit(x, *self.head, ids, teacher, temperature, d, loss_dtype=torch.float32)
        return MeanLoss.apply(self.hidden(tokens, index), call, tokens.shape[0], gain)


def batch(lengths, vocab, prompts, seed=0, device="cuda"):
    """Packed sequences, task = place mod 2: tokens, index, targets (the next token; -100 in the prompt and at the end)."""
    g = torch.Generator().manual_seed(seed)
    tokens = [torch.randint(vocab, (n,), generator=g) for n in lengths]
    target = []
    for t, p in zip(tokens, prompts):
        after = torch.cat((t[1:], torch.tensor([-100])))
        after[:p] = -100
        target.append(after)
    index = torch.cat([torch.full((n,), i % 2, dtype=torch.int32) for i, n in enumerate(lengths)])
    return torch.cat(tokens).to(device), index.to(device), torch.cat(target).to(device)


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 10
    model = Model()
    tokens, index, target = batch([40, 33, 70, 9], 512, [8, 5, 10, 2])
    optimizer = torch.optim.SGD(model.parameters(), lr=0.5)
    for step in range(steps):
        optimizer.zero_grad()
        loss = model.loss(tokens, index, target)
        loss.backward()
        optimizer.step()
        print(f"step {step}: loss {loss.item():.4f}")
    g = torch.Generator().manual_seed(1)
    ids = torch.stack([torch.randperm(512, generator=g)[:8] for _ in range(len(tokens))]).cuda()
    teacher = torch.randn(len(tokens), 8, generator=g).cuda()
    only = torch.where(index == 1, index, -1).int()
    loss = model.distill(tokens, only, ids, teacher)
    optimizer.zero_grad()
    loss.backward()
    print(f"divergence from the teacher {loss.item():.4f}")


if __name__ == "__main__":
    main()
