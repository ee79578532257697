"""Measured cases of the operators around a 4-bit key/value cache.

rotary      the position rotation of queries and keys, forward and backward
append      new keys and values rotated, quantized to 4 bits and written into
            a paged cache (the queries of the same tokens rotated in the same
            call), then the new tokens read back as the values they stand for
attention   queries over the 4-bit paged cache: single tokens, a few tokens,
            and whole chunks of a prompt

Each case has a plain form in elementary torch operations (own = False) and
the library's calls (own = True).

The cache, per page of `page` tokens and key/value head, element type `dtype`:
    k_codes  [pages, heads, page, D / 2] uint8       element 2j in the high nibble of byte j
    v_codes  [pages, heads, page / 16, D / 2, 16]    the same bytes, 16 tokens of a byte side by side
    k_scales, v_scales [pages, heads, D / bs, page]  largest magnitude of each block of bs elements
Block tables hold page numbers [B, max_pages] (-1: none); kv_len [B] counts a
sequence's tokens in the cache, the new ones included; cu_q [B + 1] are the
offsets of each sequence's new tokens among all new tokens.
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# fp32 values of the 16 codes, as the library's code_table() documents them
NF4 = [-1.0, -0.6961929202079773, -0.5250730514526367, -0.39491748809814453, -0.28444135189056396,
       -0.18477343022823334, -0.09104999154806137, 0.0, 0.07958032935857773, 0.16093017160892487,
       0.24611228704452515, 0.33791518211364746, 0.44070979952812195, 0.5626169443130493, 0.7229567170143127,
       1.0]
_FP4 = [0.0, 1 / 12, 1 / 6, 1 / 4, 1 / 3, 1 / 2, 2 / 3, 1.0]
FP4 = _FP4 + [-v for v in _FP4]


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 16: 32 query and 8 key heads, far into a long table
        {"name": "rotary decode", "op": "rotary", "tokens": 16, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "backward": False, "fused_rows": True, "max_pos": 131072, "stretch": 8.0},
        # a training batch of 4 x 4096 tokens, both halves rotated
        {"name": "rotary train forward", "op": "rotary", "tokens": 16384, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "backward": False, "fused_rows": False, "max_pos": 4096, "stretch": 1.0},
        # its gradient where pairs are neighbours, only half of each head turns, and rows are odd in number
        {"name": "rotary train backward", "op": "rotary", "tokens": 8198, "hq": 64, "hk": 8, "dim": 128, "rot": 64,
         "dtype": "fp16", "interleaved": True, "backward": True, "fused_rows": True, "max_pos": 4099, "stretch": 1.0},

        # one new token for each of 32 sequences
        {"name": "append decode", "op": "append", "batch": 32, "new": 1, "past": 8191, "ragged": 3, "hq": 32, "hk": 8,
         "dim": 128, "rot": 128, "bs": 64, "page": 16, "dtype": "bf16", "quant": "nf4", "interleaved": False, "fused_rows": True},
        # five prompts of uneven length, nothing cached before
        {"name": "append prompts", "op": "append", "batch": 5, "new": 2501, "past": 0, "ragged": 7, "hq": 64, "hk": 8,
         "dim": 128, "rot": 128, "bs": 64, "page": 64, "dtype": "bf16", "quant": "nf4", "interleaved": False, "fused_rows": True},
        # chunks that begin and end inside a page; a key head for every query head, half of it turned
        {"name": "append chunks", "op": "append", "batch": 3, "new": 1021, "past": 3333, "ragged": 11, "hq": 32, "hk": 32,
         "dim": 64, "rot": 32, "bs": 32, "page": 16, "dtype": "fp16", "quant": "fp4", "interleaved": True, "fused_rows": False},

        # the smallest call: one sequence, one token, a short context
        {"name": "decode one short", "op": "attention", "batch": 1, "new": 1, "past": 1000, "ragged": 0, "hq": 32, "hk": 8,
         "dim": 128, "bs": 64, "page": 16, "dtype": "bf16", "quant": "nf4", "window": 0},
        # a served batch of uneven contexts
        {"name": "decode batch", "op": "attention", "batch": 64, "new": 1, "past": 8191, "ragged": 5, "hq": 32, "hk": 8,
         "dim": 128, "bs": 64, "page": 64, "dtype": "bf16", "quant": "nf4", "window": 0},
        # one very long context, which has to be split to fill the GPU
        {"name": "decode one long", "op": "attention", "batch": 1, "new": 1, "past": 196610, "ragged": 0, "hq": 64, "hk": 8,
         "dim": 128, "bs": 64, "page": 64, "dtype": "bf16", "quant": "nf4", "window": 0},
        # four drafted tokens checked at once, a key head for every query head, a sliding window
        {"name": "verify drafts", "op": "attention", "batch": 24, "new": 4, "past": 9001, "ragged": 9, "hq": 32, "hk": 32,
         "dim": 64, "bs": 32, "page": 16, "dtype": "fp16", "quant": "fp4", "window": 4096},
        # three prompts of uneven length from nothing
        {"name": "prompts", "op": "attention", "batch": 3, "new": 4097, "past": 0, "ragged": 13, "hq": 32, "hk": 8,
         "dim": 128, "bs": 64, "page": 64, "dtype": "bf16", "quant": "nf4", "window": 0},
        # one chunk of a long prompt over what is cached of it: the largest
        {"name": "prompt chunk", "op": "attention", "batch": 1, "new": 2048, "past": 32768, "ragged": 0, "hq": 64, "hk": 8,
         "dim": 128, "bs": 128, "page": 128, "dtype": "bf16", "quant": "nf4", "window": 0},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention"])
    hq, hk = rng.choice([(32, 8), (64, 8), (32, 32), (16, 1), (16, 2), (12, 4), (28, 4)])
    dim = rng.choice([64, 96, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    if op == "rotary":
        c = {"op": op, "tokens": _log(rng, 1, 8192), "hq": hq, "hk": hk, "dim": dim, "rot": rot,
             "dtype": rng.choice(["bf16", "fp16", "fp32"]), "interleaved": rng.random() < 0.4, "backward": rng.random() < 0.5,
             "fused_rows": rng.random() < 0.5, "max_pos": _log(rng, 1000, 131072), "stretch": rng.choice([1.0, 4.0, 32.0])}
        c["tokens"] = max(1, min(c["tokens"], 80_000_000 // ((hq + hk) * dim * (2 if c["dtype"] == "fp32" else 1))))
        return c
    bs = rng.choice([b for b in (32, 64, 128) if dim % b == 0])
    c = {"op": op, "hq": hq, "hk": hk, "dim": dim, "bs": bs, "page": rng.choice([16, 32, 64, 128]),
         "dtype": rng.choice(["bf16", "bf16", "fp16"]), "quant": rng.choice(["nf4", "nf4", "fp4"]), "ragged": rng.randrange(1, 1000)}
    if op == "append":
        c.update(batch=_log(rng, 1, 64), past=rng.choice([0, _log(rng, 1, 8000)]), rot=rot, interleaved=rng.random() < 0.4,
                 fused_rows=rng.random() < 0.5)
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        c["new"] = max(1, min(c["new"], 40_000_000 // (c["batch"] * (hq + 2 * hk) * dim)))
        return c
    c["window"] = rng.choice([0, 0, _log(rng, 16, 4096)])
    if rng.random() < 0.6:  # single tokens, or a few
        c.update(batch=_log(rng, 1, 64), new=rng.choice([1, 1, 1, rng.randrange(2, 9)]))
        c["past"] = _log(rng, 1, max(2, min(150_000, 250_000_000 // (c["batch"] * hk * dim))))
    else:  # chunks
        c.update(batch=_log(rng, 1, 6), new=_log(rng, 9, 2048))
        c["past"] = rng.choice([0, _log(rng, 1, 24_000)])
        most = 64 * 2048 * 33792 * 128 / 2
        while c["batch"] * c["new"] * (c["past"] + c["new"]) * hq * dim > most:
            c["new"], c["past"] = max(9, c["new"] * 3 // 4), c["past"] * 3 // 4
    return c


def _lengths(case):
    """New tokens and whole length of each sequence, from the case alone."""
    if not case["ragged"]:
        return [case["new"]] * case["batch"], [case["past"] + case["new"]] * case["batch"]
    r = random.Random(case["ragged"])
    new = [case["new"] if case["new"] <= 8 else r.randint(max(1, case["new"] // 3), case["new"]) for _ in range(case["batch"])]
    past = [r.randint(case["past"] // 8, case["past"]) for _ in range(case["batch"])]
    return new, [p + n for p, n in zip(past, new)]


def _visible(case):
    """Visible (token, key) pairs, and keys that some token of their sequence sees."""
    pairs = keys = 0
    for n, length in zip(*_lengths(case)):
        w = case["window"] or length
        pairs += sum(min(length - n + i + 1, w) for i in range(n))
        keys += min(length, w + n - 1)
    return pairs, keys


def work(case):
    size = 4 if case.get("dtype") == "fp32" else 2
    hq, hk, dim = case["hq"], case["hk"], case["dim"]
    if case["op"] == "rotary":
        n = case["tokens"] * (hq + hk)
        rows = min(case["tokens"], case["max_pos"])
        return {"bytes": 2 * n * dim * size + rows * case["rot"] * 4 + 8 * case["tokens"], "flops": n * case["rot"] * 3}
    held = dim / 2 + dim // case["bs"] * 2  # bytes of a cached row
    new, length = _lengths(case)
    if case["op"] == "append":
        t = sum(new)
        values = t * dim * 2 * (2 * hq + 4 * hk)  # q in and out, k and v in and read back
        return {"bytes": values + 4 * t * hk * held + t * case["rot"] * 4, "flops": t * (3 * (hq + hk) * case["rot"] + 8 * hk * dim)}
    pairs, keys = _visible(case)
    return {"bytes": 2 * sum(new) * hq * dim * 2 + keys * hk * 2 * held, "flops": 4 * pairs * hq * dim}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(g, tokens, heads, dim, dtype):
    """Activations [tokens, heads, dim]: unit normal, some channels stronger, as projections give them."""
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda")
    return (x * (1 + 3 * (torch.rand(heads, dim, generator=g, device="cuda") > 0.97))).to(DT[dtype])


def _qkv(g, case, tokens, parts):
    """The heads of each part, as views of one projection's rows or as tensors of their own."""
    rows = [_rows(g, tokens, h, case["dim"], case["dtype"]) for h in parts]
    return list(torch.cat(rows, 1).split(parts, 1)) if case["fused_rows"] else rows


def _rope_table(max_pos, rot, stretch):
    """cos and sin of position * 10000^(-2i / rot) / stretch, [max_pos, rot / 2, 2] in fp32."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot) / stretch
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def _code_values(quant):
    return torch.tensor(NF4 if quant == "nf4" else FP4, device="cuda")


def _paged(case, length, g):
    """A block table over pages in shuffled order, -1 where a sequence needs none."""
    need = [-(-n // case["page"]) for n in length]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(length), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "rotary":
        t = case["tokens"]
        q, k = _qkv(g, case, t, [case["hq"], case["hk"]])
        pos = torch.randint(case["max_pos"], (t,), generator=g, device="cuda") if t < 64 else torch.arange(t, device="cuda") % case["max_pos"]
        return {"case": case, "q": q, "k": k, "positions": pos, "table": _rope_table(case["max_pos"], case["rot"], case["stretch"])}
    new, length = _lengths(case)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    pages, table = _paged(case, length, g)
    s = {"case": case, "block_table": table, "kv_len": torch.tensor(length, **i32), "cu_q": torch.tensor(cu, **i32),
         "max_q": max(new), "max_kv": max(length), "pages": pages}
    hk, dim, page, bs, dtype = case["hk"], case["dim"], case["page"], case["bs"], DT[case["dtype"]]
    if case["op"] == "append":
        s["k_codes"] = torch.zeros(pages, hk, page, dim // 2, dtype=torch.uint8, device="cuda")
        s["v_codes"] = torch.zeros(pages, hk, page // 16, dim // 2, 16, dtype=torch.uint8, device="cuda")
        s["k_scales"] = torch.zeros(pages, hk, dim // bs, page, dtype=dtype, device="cuda")
        s["v_scales"] = torch.zeros_like(s["k_scales"])
        s["q"], s["k"], s["v"] = _qkv(g, case, cu[-1], [case["hq"], hk, hk])
        s["table"] = _rope_table(max(length), case["rot"], 1.0)
        return s
    # what an earlier part of the sequences left in the cache: quantized normal rows, page by page
    for name in ("k", "v"):
        codes, scales = [], []
        step = max(1, (1 << 25) // (hk * page * dim))
        gain = 1 + 3 * (torch.rand(hk, 1, dim, generator=g, device="cuda") > (0.97 if name == "k" else 2))
        for p in range(0, pages, step):
            x = (torch.randn(min(step, pages - p), hk, page, dim, generator=g, device="cuda") * gain).to(dtype)
            c, a = _encode(x, bs, case["quant"])
            codes.append(c)
            scales.append(a.transpose(-1, -2).to(dtype))
        codes = torch.cat(codes)
        if name == "v":
            codes = codes.view(pages, hk, page // 16, 16, dim // 2).transpose(-1, -2).contiguous()
        s[name + "_codes"], s[name + "_scales"] = codes, torch.cat(scales).contiguous()
    s["q"] = torch.randn(cu[-1], case["hq"], dim, generator=g, device="cuda").to(dtype)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _rotate(x, cs, interleaved, backward=False):
    """x [T, H, D] with its first 2 * cs.shape[1] elements turned by cs [T, rot / 2, 2], in fp32."""
    x = x.float()
    half = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if backward:
        s = -s
    part, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :half], part[..., half:]
    u, w = a * c - b * s, b * c + a * s
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, rest), -1)


def _encode(x, bs, quant):
    """Nearest codes [..., D / 2] packed two to a byte, and block maxima [..., D / bs], of x [..., D]."""
    x = x.float().unflatten(-1, (-1, bs))
    a = x.abs().amax(-1)
    if quant == "nf4":
        t = torch.tensor(NF4, device=x.device)
        above = x[..., None] > a[..., None, None] * ((t[1:] + t[:-1]) / 2)
        at0 = x[..., None] >= a[..., None, None] * ((t[1:8] + t[:7]) / 2)  # ties go to the smaller magnitude
        code = at0.sum(-1) + above[..., 7:].sum(-1)
        code = torch.where(a[..., None] > 0, code, 7)
    else:
        t = torch.tensor(FP4[:8], device=x.device)
        code = (x.abs()[..., None] > a[..., None, None] * ((t[1:] + t[:-1]) / 2)).sum(-1)
        code = torch.where((x < 0) & (code > 0), code + 8, code)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] << 4 | code[..., 1::2], a


def _values(codes, scales, quant):
    """fp32 values [..., D] of packed codes [..., D / 2] with block scales [..., D / bs]."""
    t = _code_values(quant)
    x = torch.stack((t[(codes >> 4).int()], t[(codes & 15).int()]), -1).flatten(-2)
    return (x.unflatten(-1, (scales.shape[-1], -1)) * scales.float()[..., None]).flatten(-2)


def _token_places(s, tokens):
    """For each new token: its sequence, its place among the sequence's new tokens, its position."""
    t = torch.arange(tokens, device="cuda")
    seq = (t[:, None] >= s["cu_q"][None, 1:]).sum(1)
    first = s["cu_q"][:-1].long()
    i = t - first[seq]
    n = s["cu_q"][1:].long() - first
    return seq, i, s["kv_len"].long()[seq] - n[seq] + i


def _plain_append(s):
    c = s["case"]
    seq, _, pos = _token_places(s, s["k"].shape[0])
    cs = s["table"][pos]
    dtype = s["k"].dtype
    q = _rotate(s["q"], cs, c["interleaved"]).to(dtype)
    k = _rotate(s["k"], cs, c["interleaved"]).to(dtype)  # the cache's element type: what is quantized
    page = s["block_table"][seq, pos // c["page"]].long()
    at = pos % c["page"]
    back = []
    for_v = s["v_codes"].view(s["pages"], c["hk"], -1, c["dim"] // 2, 16)
    kc, ka = _encode(k, c["bs"], c["quant"])
    vc, va = _encode(s["v"], c["bs"], c["quant"])
    s["k_codes"][page, :, at] = kc
    for_v[page, :, at // 16, :, at % 16] = vc
    s["k_scales"][page, :, :, at] = ka.to(dtype)
    s["v_scales"][page, :, :, at] = va.to(dtype)
    back.append(_values(s["k_codes"][page, :, at], s["k_scales"][page, :, :, at], c["quant"]).to(dtype))
    back.append(_values(for_v[page, :, at // 16, :, at % 16], s["v_scales"][page, :, :, at], c["quant"]).to(dtype))
    return [q] + back


def _cached(s):
    """K and V of every sequence in fp32, [B, heads, max_pages * page, D]."""
    c = s["case"]
    bt = s["block_table"].clamp(min=0).long()
    k = _values(s["k_codes"][bt], s["k_scales"][bt].transpose(-1, -2), c["quant"])
    vc = s["v_codes"][bt].transpose(-1, -2).flatten(3, 4)
    v = _values(vc, s["v_scales"][bt].transpose(-1, -2), c["quant"])
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    c, q = s["case"], s["q"]
    tokens, hq, dim = q.shape
    group = hq // c["hk"]
    k, v = _cached(s)
    batch, _, keys, _ = k.shape
    first, n = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(s["max_q"], device="cuda")
    x = q.float()[(first[:, None] + i).clamp(max=tokens - 1)]  # [B, max_q, hq, D]
    x = x.view(batch, s["max_q"], c["hk"], group, dim).permute(0, 2, 3, 1, 4).reshape(batch, c["hk"], -1, dim)
    score = torch.matmul(x, k.transpose(-1, -2).contiguous()) * dim ** -0.5
    score = score.view(batch, c["hk"], group, s["max_q"], keys)
    pos = (s["kv_len"].long() - n)[:, None] + i  # [B, max_q]
    j = torch.arange(keys, device="cuda")
    seen = j <= pos[..., None]
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(batch, c["hk"], -1, keys), v).view(batch, c["hk"], group, s["max_q"], dim)
    out = torch.where(total > 0, out / total, 0.0)
    seq, i, _ = _token_places(s, tokens)
    return out.permute(0, 3, 1, 2, 4).reshape(batch, s["max_q"], hq, dim)[seq, i].to(q.dtype)


# --------------------------------------------------------------------------
def _handle(s):
    """The library's view of the cache, made once as a user's program keeps it."""
    if "handle" not in s:
        import quantized_matvec_amd as qmv
        s["qmv"] = qmv
        s["handle"] = qmv.KVCache4bit.from_tensors(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["case"]["quant"])
    return s["qmv"], s["handle"]


def run(s):
    c = s["case"]
    if c["op"] == "rotary":
        if own:
            import quantized_matvec_amd as qmv
            turn = qmv.rotary_backward if c["backward"] else qmv.rotary
            return turn(s["q"], s["k"], s["table"], s["positions"], interleaved=c["interleaved"])
        cs = s["table"][s["positions"]]
        return [_rotate(x, cs, c["interleaved"], c["backward"]).to(x.dtype) for x in (s["q"], s["k"])]
    one = s["max_q"] == 1
    if c["op"] == "append":
        if not own:
            return _plain_append(s)
        qmv, cache = _handle(s)
        cu = None if one else s["cu_q"]
        q = qmv.kv_append_4bit(cache, s["k"], s["v"], s["block_table"], s["kv_len"], cu_q=cu, max_q=s["max_q"], q=s["q"],
                               table=s["table"], interleaved=c["interleaved"])
        k, v = qmv.kv_dequantize_4bit(cache, s["block_table"], s["kv_len"], s["k"].shape[0], cu_q=cu, max_q=s["max_q"])
        return [q, k, v]
    if not own:
        return _plain_attention(s)
    qmv, cache = _handle(s)
    return qmv.attention_4bit(s["q"], cache, s["block_table"], s["kv_len"], cu_q=None if one else s["cu_q"], max_q=s["max_q"],
                              max_kv=s["max_kv"], window=c["window"])


# --------------------------------------------------------------------------
# the definitions in 64 bits, token by token and sequence by sequence
# --------------------------------------------------------------------------
def _turn64(x, cs, interleaved, backward):
    half = cs.shape[1]
    rot = torch.complex(cs[..., 0].double(), (-1.0 if backward else 1.0) * cs[..., 1].double())[:, None]
    out = x.double().clone()
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.complex(out[..., first], out[..., second]) * rot
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _nearest64(x, bs, quant):
    """x [..., D] after its 4-bit form: the nearest code value times the block's largest magnitude."""
    t = torch.tensor(sorted(set(NF4 if quant == "nf4" else FP4), key=abs), device=x.device).double()  # a tie takes the smaller magnitude
    shape = x.shape
    x = x.double().reshape(-1, bs)
    out = torch.empty_like(x)
    for at in range(0, x.shape[0], 1 << 17):
        y = x[at:at + (1 << 17)]
        a = y.abs().amax(1, keepdim=True)
        off = (y[..., None] - a[..., None] * t).abs()
        out[at:at + (1 << 17)] = t[off.argmin(-1)] * a
    return out.view(shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        cs = s["table"][s["positions"]]
        return [_turn64(x, cs, case["interleaved"], case["backward"]) for x in (s["q"], s["k"])]
    new, length = _lengths(case)
    if case["op"] == "append":
        pos = torch.cat([torch.arange(m - n, m, device="cuda") for n, m in zip(new, length)])
        cs = s["table"][pos]
        k = _turn64(s["k"], cs, case["interleaved"], False).to(s["k"].dtype)
        return [_turn64(s["q"], cs, case["interleaved"], False), _nearest64(k, case["bs"], case["quant"]),
                _nearest64(s["v"], case["bs"], case["quant"])]
    group, dim = case["hq"] // case["hk"], case["dim"]
    t = _code_values(case["quant"]).double()
    out, at = [], 0
    for b, (n, m) in enumerate(zip(new, length)):
        pages = s["block_table"][b, :-(-m // case["page"])].long()
        heads = []
        for h in range(case["hk"]):
            kv = []
            for name in ("k", "v"):
                codes = s[name + "_codes"][pages, h]
                if name == "v":
                    codes = codes.permute(0, 1, 3, 2)
                codes = codes.reshape(-1, dim // 2)[:m]
                x = torch.empty(m, dim, dtype=torch.float64, device="cuda")
                x[:, 0::2], x[:, 1::2] = t[(codes // 16).long()], t[(codes % 16).long()]
                scales = s[name + "_scales"][pages, h].double().permute(0, 2, 1).reshape(-1, dim // case["bs"])[:m]
                kv.append(x * scales.repeat_interleave(case["bs"], 1))
            pos = torch.arange(m - n, m, device="cuda")[:, None]
            j = torch.arange(m, device="cuda")[None]
            hidden = (j > pos) | ((j <= pos - case["window"]) if case["window"] else False)
            for u in range(h * group, (h + 1) * group):
                score = s["q"][at:at + n, u].double() @ kv[0].t() / dim ** 0.5
                heads.append(score.masked_fill_(hidden, float("-inf")).softmax(-1) @ kv[1])
        out.append(torch.stack(heads, 1))
        at += n
    return torch.cat(out)
