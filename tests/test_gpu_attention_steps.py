"""The division of attention_4bit's work: every key of a row counts once.

All weights are equal (queries of zeros) and a cached value is 1 in one
element, that of its step of 64 keys modulo the head size, and 0 elsewhere:
the result counts, exactly, the keys of each step.  A step that is lost, taken
twice or added to another row shifts an element by a tenth or more, a single
key by more than fp16's rounding (bfloat16's hides it, but not a step)."""
import numpy as np
import pytest
import torch

from quantized_matvec_amd import KVCache4bit, attention_4bit

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
ZERO, ONE = 7, 15       # NF4 codes
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def counting_cache(lens, hk, dim, page, dt):
    """Sequences whose token j, head h has its 1 at element (j // 64 + h) % dim."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = np.random.default_rng(sum(lens)).permutation(pages)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    codes = np.full((pages, hk, page, dim), ONE, np.uint8)     # what belongs to no token: ones
    at = 0
    for b, n in enumerate(lens):
        for i in range(need[b]):
            p = table[b, i] = order[at]
            at += 1
            j = np.arange(i * page, min((i + 1) * page, n))
            codes[p, :, :len(j)] = ZERO
            for h in range(hk):
                codes[p, h, j - i * page, (j // 64 + h) % dim] = ONE
    packed = codes[..., 0::2] << 4 | codes[..., 1::2]
    vc = np.ascontiguousarray(packed.reshape(pages, hk, page // 16, 16, dim // 2).swapaxes(-1, -2))
    scales = torch.ones(pages, hk, 1 if dim & (dim - 1) == 0 else dim // 32, page, dtype=dt, device="cuda")
    kc = torch.randint(0, 256, packed.shape, dtype=torch.uint8, device="cuda")
    return KVCache4bit.from_tensors(kc, scales, torch.from_numpy(vc).cuda(), scales.clone()), torch.from_numpy(table).cuda()


def check(lens, new, hq, hk, dim, page=64, window=0, causal=True, max_kv=None, dt=torch.float16):
    cache, table = counting_cache(lens, hk, dim, page, dt)
    cu = [0] + np.cumsum(new).tolist()
    q = torch.zeros(cu[-1], hq, dim, dtype=dt, device="cuda")
    got = attention_4bit(q, cache, table, i32(lens), cu_q=i32(cu), max_q=max(new), window=window, causal=causal, max_kv=max_kv)
    got = got.double().cpu().numpy()
    G = hq // hk
    for b, n in enumerate(new):
        pos = lens[b] - n + np.arange(n)
        hi = np.maximum(np.minimum(pos + 1, lens[b]) if causal else np.full(n, lens[b]), 0)
        lo = np.maximum(pos - window + 1, 0) if window else np.zeros(n, int)
        for h in range(hk):
            where = (np.arange(max(lens[b], 1)) // 64 + h) % dim
            sums = np.zeros((n, dim))
            for i in range(n):
                if hi[i] > lo[i]:
                    sums[i] = np.bincount(where[lo[i]:hi[i]], minlength=dim) / (hi[i] - lo[i])
            # fp32 sums of up to some 640 products of 1 (and of the factor of the code table), one rounding
            bad = np.abs(got[cu[b]:cu[b + 1], h * G:(h + 1) * G] - sums[:, None]) > (U[dt] + 2.0 ** -14) * sums[:, None]
            assert not bad.any(), (b, h, np.argwhere(bad)[:4].tolist())


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 1), (8, 2), (12, 4), (16, 1), (3, 3)])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_single_tokens(hq, hk, dim):
    check([40000], [1], hq, hk, dim)
    check([9000, 1, 64, 700, 12000, 65, 3, 4097, 0, 511], [1] * 10, hq, hk, dim, 16)
    check([30011, 12, 9000], [1] * 3, hq, hk, dim, 128, window=4097)


@pytest.mark.parametrize("hq,hk,new", [(4, 1, [4, 1, 3, 0]), (32, 4, [2, 2, 1, 1]), (8, 8, [17, 33, 48, 16]), (34, 2, [2, 0, 1, 1])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_few_tokens(hq, hk, new, dim):
    check([20000, 77, 4100, 640], new, hq, hk, dim)
    check([20000, 77, 4100, 640], new, hq, hk, dim, 16, window=1000)
    check([20000, 77, 4100, 640], new, hq, hk, dim, 32, causal=False, max_kv=20000)


@pytest.mark.parametrize("hq,hk,new", [(4, 1, [64, 1, 13]), (8, 2, [200, 0, 300]), (1, 1, [257, 256, 1])])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_prompts(hq, hk, new, dim, dt):
    check([17000, 77, 400], new, hq, hk, dim, dt=dt)
    check([17000, 77, 400], new, hq, hk, dim, 16, window=1000, dt=dt)
    check([17000, 77, 400], new, hq, hk, dim, 128, causal=False, dt=dt)


@pytest.mark.parametrize("hq,hk,dim", [(8, 2, 128), (4, 4, 64), (16, 1, 256)])
@pytest.mark.parametrize("prompt", [13, 64, 700])
def test_prompts_and_single_tokens_together(hq, hk, dim, prompt):
    """One prompt among the single tokens of long sequences."""
    lens = [9000, 1, 4097, 64, 12000, 333, 6000, 2049, 8191, 700 + prompt, 1023, 17, 5000, 8, 16000, 2]
    new = [1] * 9 + [prompt] + [1] * 6
    check(lens, new, hq, hk, dim)
    check(lens, new, hq, hk, dim, 16, window=3000)


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("dim", [32, 160, 224])
def test_other_head_sizes(dim, new):
    check([3000, 77], [new, 1], 4, 2, dim)
    check([3000, 77], [new, 1], 4, 2, dim, 16, window=300)


def test_every_length():
    """Around each border of a step, of a wave's and of a workgroup's run."""
    for lens in (list(range(1, 200)), [64 * n + d for n in range(1, 70, 3) for d in (-1, 0, 1)]):
        check(lens, [1] * len(lens), 2, 1, 64, 16)
