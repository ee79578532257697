"""A small decoder whose weights and key/value cache are all held in 4 bits.

Random weights, 2 layers: embedding_4bit -> (gemm_4bit projections ->
kv_append_4bit with the position rotation -> attention_4bit -> gemm_4bit
output) and a gated MLP per layer -> gemm_4bit logits.  Two prompts of uneven
length are taken in at once, then tokens are generated one by one for both
sequences out of one paged cache.

    python examples/decoder_4bit.py [tokens]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matvec_amd as qmv  # noqa: E402
from quantized_matvec_amd.qmv import embedding_4bit  # noqa: E402


class Decoder4bit:
    def __init__(self, vocab=512, width=512, layers=2, q_heads=8, kv_heads=2, head_dim=64, mlp=1024,
                 pages=64, page_size=16, max_pos=1024, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        weight = lambda n, k: qmv.quantize_4bit(
            (torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(dtype), 64, "nf4", double_quant=True)
        self.heads, self.kv_heads, self.dim, self.dtype, self.device = q_heads, kv_heads, head_dim, dtype, device
        self.embedding = weight(vocab, width)
        self.layers = [dict(qkv=weight((q_heads + 2 * kv_heads) * head_dim, width), out=weight(width, q_heads * head_dim),
                            up=weight(2 * mlp, width), down=weight(width, mlp)) for _ in range(layers)]
        self.logits = weight(vocab, width)
        self.caches = [qmv.KVCache4bit(pages, kv_heads, page_size, head_dim, 64, "nf4", dtype, device)
                       for _ in range(layers)]
        self.rope = qmv.rope_table(qmv.rope_frequencies(head_dim), max_pos, device=device)

    def linear(self, x, name):
        packed, state = name
        return qmv.gemv_4bit(x, packed, state) if x.shape[0] <= 8 else qmv.gemm_4bit(x, packed, state)

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)

    def step(self, tokens, block_table, kv_len, cu_q=None, max_q=1):
        """Logits [tokens, vocab] of new tokens, whose keys and values join the caches."""
        x = embedding_4bit(tokens, *self.embedding, out_dtype=self.dtype)
        n = x.shape[0]
        for layer, cache in zip(self.layers, self.caches):
            qkv = self.linear(self.norm(x), layer["qkv"]).view(n, -1, self.dim)
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)  # views: taken as they are
            q = qmv.kv_append_4bit(cache, k, v, block_table, kv_len, cu_q, max_q, q=q, table=self.rope)
            y = qmv.attention_4bit(q, cache, block_table, kv_len, cu_q, max_q)
            x = x + self.linear(y.reshape(n, -1), layer["out"])
            gate, up = self.linear(self.norm(x), layer["up"]).chunk(2, -1)
            x = x + self.linear((torch.nn.functional.silu(gate) * up).contiguous(), layer["down"])
        return self.linear(self.norm(x), self.logits)


def tables(model, lengths, room):
    """Pages for sequences of these lengths with `room` tokens to come."""
    page = model.caches[0].page_size
    need = [-(-(n + room) // page) for n in lengths]
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    return table.to(model.device)


def generate(model, prompts, count):
    """Greedy continuations [len(prompts)][count] and the logits of every step."""
    i32 = dict(dtype=torch.int32, device=model.device)
    lengths = [len(p) for p in prompts]
    table = tables(model, lengths, count)
    kv_len = torch.tensor(lengths, **i32)
    cu = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), **i32)
    logits = model.step(torch.cat(prompts).to(model.device), table, kv_len, cu, max(lengths))
    logits = logits[(cu[1:] - 1).long()]           # each prompt's last token
    steps, tokens = [logits], [logits.argmax(-1)]
    for _ in range(count - 1):
        kv_len += 1
        logits = model.step(tokens[-1], table, kv_len)
        steps.append(logits)
        tokens.append(logits.argmax(-1))
    return torch.stack(tokens, 1), torch.stack(steps, 1)


def main():
    count = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    model = Decoder4bit()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(512, (n,), generator=g) for n in (37, 5)]
    tokens, _ = generate(model, prompts, count)
    for p, t in zip(prompts, tokens.tolist()):
        print(f"prompt of {len(p)} tokens -> {t}")
    held = sum(c.nbytes for c in model.caches)
    print(f"caches: {held} bytes for {model.caches[0].num_pages * model.caches[0].page_size} tokens and {len(model.caches)} layers")


if __name__ == "__main__":
    main()
