"""Measured cases of the operators of fine-tuning over frozen 4-bit weights.

lora           a 4-bit projection with the low-rank adapters of many requests beside it
lora_backward  its gradients: inputs, and every adapter's two factors
cross_entropy  softmax cross entropy over a 4-bit vocabulary projection, with or without the gradient of its inputs
distill        the divergence from a teacher's top logits over the same projection, likewise

Each case has a plain form in elementary torch operations (own = False) and
the library's calls (own = True).

A weight [rows, K] is held as `packed` [rows * K / 2] uint8, element 2j in the
high nibble of byte j, and one scale for each block of `bs` elements: fp32, or
8-bit codes of (scale - offset) in groups of 256 with an fp32 scale each.
Adapters are stacks A [n, R, K] and B [n, N, R] with a scale [n]; index [T]
says which one a token uses (-1: none).
"""
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

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
        # one token of one request through an attention-sized projection
        {"name": "lora one token", "op": "lora", "tokens": 1, "requests": 1, "n": 1, "rank": 16, "N": 4096, "K": 4096,
         "bs": 64, "quant": "nf4", "double": True, "dtype": "bf16", "bias": False, "ragged": 0},
        # a decode step of 32 requests, each with a fine-tune of its own
        {"name": "lora decode", "op": "lora", "tokens": 32, "requests": 32, "n": 48, "rank": 16, "N": 14336, "K": 4096,
         "bs": 64, "quant": "nf4", "double": True, "dtype": "bf16", "bias": False, "ragged": 1},
        # short prompts of a few requests, one of them without an adapter; an odd number of rows, and a bias
        {"name": "lora short prompts", "op": "lora", "tokens": 301, "requests": 5, "n": 7, "rank": 64, "N": 8192, "K": 2048,
         "bs": 32, "quant": "fp4", "double": False, "dtype": "fp16", "bias": True, "ragged": 2},
        # long prompts of eight requests, packed
        {"name": "lora prompts", "op": "lora", "tokens": 4099, "requests": 8, "n": 8, "rank": 32, "N": 14336, "K": 4096,
         "bs": 64, "quant": "nf4", "double": True, "dtype": "bf16", "bias": False, "ragged": 3},

        # a training step's batch through the same projection: one adapter
        {"name": "lora train", "op": "lora_backward", "tokens": 4096, "requests": 1, "n": 1, "rank": 16, "N": 14336, "K": 4096,
         "bs": 64, "quant": "nf4", "double": True, "dtype": "bf16", "bias": False, "ragged": 0},
        # several adapters trained at once on uneven shares of an odd batch, down projection
        {"name": "lora train several", "op": "lora_backward", "tokens": 1537, "requests": 9, "n": 4, "rank": 64, "N": 4096, "K": 14336,
         "bs": 128, "quant": "fp4", "double": False, "dtype": "fp16", "bias": False, "ragged": 5},

        # a few answers scored: the loss alone
        {"name": "score few", "op": "cross_entropy", "tokens": 17, "vocab": 32000, "K": 2048, "bs": 64, "quant": "nf4",
         "double": True, "dtype": "bf16", "grad": False, "ignore": 0.0},
        # held-out text scored
        {"name": "score text", "op": "cross_entropy", "tokens": 2048, "vocab": 128256, "K": 4096, "bs": 64, "quant": "nf4",
         "double": True, "dtype": "bf16", "grad": False, "ignore": 0.0},
        # an odd vocabulary and an odd batch
        {"name": "train odd vocabulary", "op": "cross_entropy", "tokens": 1023, "vocab": 50257, "K": 1024, "bs": 64, "quant": "nf4",
         "double": False, "dtype": "fp16", "grad": True, "ignore": 0.1},
        # a training batch whose prompts do not count: the largest
        {"name": "train answers", "op": "cross_entropy", "tokens": 4096, "vocab": 128256, "K": 4096, "bs": 64, "quant": "nf4",
         "double": True, "dtype": "bf16", "grad": True, "ignore": 0.3},

        # a short batch against eight kept logits of each token
        {"name": "distill short", "op": "distill", "tokens": 96, "vocab": 32003, "K": 2048, "bs": 64, "quant": "nf4", "double": False,
         "dtype": "fp16", "grad": True, "k": 8, "tau": 2.0, "short": 0.2},
        # a training batch against the teacher's 64 largest logits
        {"name": "distill", "op": "distill", "tokens": 2048, "vocab": 128256, "K": 4096, "bs": 64, "quant": "nf4", "double": True,
         "dtype": "bf16", "grad": True, "k": 64, "tau": 1.0, "short": 0.05},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_backward", "cross_entropy", "cross_entropy", "distill"])
    c = {"op": op, "bs": rng.choice([32, 64, 64, 128]), "quant": rng.choice(["nf4", "nf4", "fp4"]), "double": rng.random() < 0.5,
         "dtype": rng.choice(["bf16", "bf16", "fp16"])}
    K = c["bs"] * _log(rng, 512 // c["bs"], 8192 // c["bs"])
    if op.startswith("lora"):
        c.update(N=32 * _log(rng, 16, 448), K=K, rank=rng.choice([8, 16, 16, 32, 64, 128]), n=_log(rng, 1, 48),
                 bias=op == "lora" and rng.random() < 0.3, ragged=rng.randrange(1, 1000))
        c["tokens"] = _log(rng, 1, 4096) if op == "lora" else _log(rng, 16, 4096)
        c["tokens"] = max(1, min(c["tokens"], 4096 * 14336 * 4096 // (c["N"] * K)))
        c["requests"] = c["tokens"] if c["tokens"] <= 64 else _log(rng, 1, 64)
        return c
    c.update(tokens=_log(rng, 1, 4096), vocab=_log(rng, 1000, 128256), K=K, grad=rng.random() < 0.6)
    c["tokens"] = max(1, min(c["tokens"], 2048 * 128256 * 4096 // (c["vocab"] * K)))
    if op == "cross_entropy":
        c["ignore"] = rng.choice([0.0, 0.0, 0.1, 0.5])
    else:
        c.update(k=_log(rng, 1, 128), tau=rng.choice([1.0, 1.0, 2.0, 4.0]), short=rng.choice([0.0, 0.1]))
    return c


def _index(case):
    """The adapter of every token, from the case alone: requests one after the other, some without an adapter."""
    r = random.Random(case["ragged"])
    T, q = case["tokens"], case["requests"]
    if q == 1:
        return [0] * T
    cuts = sorted(r.randrange(T + 1) for _ in range(q - 1)) if q < T else list(range(1, T))
    of = [r.randrange(case["n"]) if r.random() < 0.9 else -1 for _ in range(q)]
    out = []
    for a, lo, hi in zip(of, [0] + cuts, cuts + [T]):
        out += [a] * (hi - lo)
    return out


def _held(case, rows):
    blocks = rows * case["K"] // case["bs"]
    return rows * case["K"] / 2 + (blocks + 4 * (blocks / 256) if case["double"] else 4 * blocks)


def work(case):
    T, K = case["tokens"], case["K"]
    if case["op"].startswith("lora"):
        index, N, R = _index(case), case["N"], case["rank"]
        used, active = len(set(index) - {-1}), sum(a >= 0 for a in index)
        moved = 2 * T * (K + N) + _held(case, N) + 2 * used * R * (K + N)
        if case["op"] == "lora":
            return {"bytes": moved + 4 * T, "flops": 2 * T * N * K + 2 * active * R * (K + N)}
        # x and dy read, dx and all adapters' gradients written
        return {"bytes": moved + 4 * T + 2 * T * K + 2 * case["n"] * R * (K + N), "flops": 2 * T * N * K + 2 * active * R * (2 * N + 3 * K)}
    V = case["vocab"]
    live = T * (1 - case.get("ignore", 0.0))  # a token whose target does not count needs no logits
    k = case.get("k", 1)
    return {"bytes": 2 * live * K + _held(case, V) + T * (8 * k + 2) + (4 * T * k if case["op"] == "distill" else 0) + (2 * T * K + 4 * T if case["grad"] else 0),
            "flops": (4 if case["grad"] else 2) * live * V * K}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weight(g, case, rows, gain):
    """A quantized weight of about gain / sqrt(K) standard deviation.  The codes of
    a quantized normal weight are used about evenly, its scales vary little."""
    n, K = rows * case["K"], case["K"]
    blocks = n // case["bs"]
    packed = torch.randint(256, (n // 2,), generator=g, device="cuda", dtype=torch.uint8)
    unit = gain * K ** -0.5 / 0.55
    if not case["double"]:
        return {"packed": packed, "absmax": unit * (0.7 + 0.6 * torch.rand(blocks, generator=g, device="cuda"))}
    return {"packed": packed, "absmax_q": torch.randint(256, (blocks,), generator=g, device="cuda", dtype=torch.uint8),
            "absmax2": unit * (0.2 + 0.2 * torch.rand(-(-blocks // 256), generator=g, device="cuda")),
            "offset": torch.full((1,), unit, device="cuda"),
            "code2": ((torch.arange(256, dtype=torch.float64) - 127) / 127).float().cuda()}


def _rows(g, tokens, width, dtype):
    """Activations: unit normal, some channels stronger, as a norm before a projection gives them."""
    x = torch.randn(tokens, width, generator=g, device="cuda")
    return (x * (1 + 2 * (torch.rand(width, generator=g, device="cuda") > 0.98))).to(DT[dtype])


def prepare(case, seed):
    g = _gen(seed)
    T, K, dtype = case["tokens"], case["K"], DT[case["dtype"]]
    if case["op"].startswith("lora"):
        N, R, n = case["N"], case["rank"], case["n"]
        s = {"case": case, "rows": N, **_weight(g, case, N, 1.0), "x": _rows(g, T, K, case["dtype"])}
        s["index"] = torch.tensor(_index(case), dtype=torch.int32, device="cuda")
        s["A"] = (torch.randn(n, R, K, generator=g, device="cuda") * K ** -0.5).to(dtype)
        s["B"] = (torch.randn(n, N, R, generator=g, device="cuda") * 0.3 * R ** -0.5).to(dtype)
        s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        s["bias"] = torch.randn(N, generator=g, device="cuda").to(dtype) if case["bias"] else None
        if case["op"] == "lora_backward":
            s["dy"] = (torch.randn(T, N, generator=g, device="cuda") * 0.01).to(dtype)
        return s
    V = case["vocab"]
    s = {"case": case, "rows": V, **_weight(g, case, V, 1.5), "x": _rows(g, T, K, case["dtype"])}
    if case["grad"]:
        # the mean over the batch, with a weight for each token; brought into the 16-bit types' range by a loss scale
        s["dloss"] = (64.0 / T) * (0.5 + torch.rand(T, generator=g, device="cuda"))
    if case["op"] == "cross_entropy":
        s["target"] = torch.randint(V, (T,), generator=g, device="cuda")
        s["target"][torch.rand(T, generator=g, device="cuda") < case["ignore"]] = -100
        return s
    # the teacher's k largest logits in falling order, fewer of them for some tokens
    k = case["k"]
    start = torch.randint(V, (T, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, V // k), (T, 1), generator=g, device="cuda")
    s["ids"] = (start + step * torch.arange(k, device="cuda")) % V
    keep = torch.where(torch.rand(T, 1, generator=g, device="cuda") < case["short"], torch.randint(k + 1, (T, 1), generator=g, device="cuda"), k)
    s["ids"] = torch.where(torch.arange(k, device="cuda") < keep, s["ids"], -1)
    s["teacher"] = (8 + 3 * torch.randn(T, k, generator=g, device="cuda")).sort(-1, descending=True)[0].to(dtype)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _weight32(s):
    """The weight [rows, K] in fp32."""
    c = s["case"]
    t = torch.tensor(NF4 if c["quant"] == "nf4" else FP4, device="cuda")
    if c["double"]:
        blocks = s["absmax_q"].numel()
        a = s["code2"][s["absmax_q"].int()] * s["absmax2"].repeat_interleave(256)[:blocks] + s["offset"]
    else:
        a = s["absmax"]
    pairs = torch.stack((t[(s["packed"] >> 4).int()], t[(s["packed"] & 15).int()]), -1)
    return (pairs.view(-1, c["bs"]) * a[:, None]).view(s["rows"], c["K"])


def _own_columns(s):
    """[T, n * R]: the scale of the token's adapter in that adapter's columns, 0 in all others."""
    n, R = s["case"]["n"], s["case"]["rank"]
    mine = (s["index"][:, None] == torch.arange(n, device="cuda")) * s["scale"]
    return mine.repeat_interleave(R, 1)


def _plain_lora(s):
    w = _weight32(s)
    x = s["x"].float()
    n, R, K = s["A"].shape
    down = s["A"].float().view(n * R, K)
    up = s["B"].float().transpose(0, 1).reshape(s["rows"], n * R)
    mine = _own_columns(s)
    u = torch.matmul(x, down.t()) * mine
    if s["case"]["op"] == "lora":
        y = torch.matmul(x, w.t()) + torch.matmul(u, up.t())
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y.to(s["x"].dtype)
    dy = s["dy"].float()
    v = torch.matmul(dy, up) * mine
    dx = torch.matmul(dy, w) + torch.matmul(v, down)
    da = torch.matmul(v.t(), x).view(n, R, K)
    db = torch.matmul(dy.t(), u).view(s["rows"], n, R).transpose(0, 1).contiguous()
    dtype = s["x"].dtype
    return [dx.to(dtype), da.to(dtype), db.to(dtype)]


def _plain_loss(s):
    c, x = s["case"], s["x"]
    w = _weight32(s)
    tau = c.get("tau", 1.0)
    logits = torch.matmul(x.float(), w.t()) / tau
    top = logits.amax(-1, keepdim=True)
    lse = top + (logits - top).exp().sum(-1, keepdim=True).log()
    if c["op"] == "cross_entropy":
        ids, there = s["target"][:, None], (s["target"] >= 0)[:, None]
        p, logp = there.float(), torch.zeros_like(lse)
    else:
        ids, there = s["ids"], s["ids"] >= 0
        z = (s["teacher"].float() / tau).masked_fill(~there, float("-inf"))
        high = z.amax(-1, keepdim=True).clamp(min=-3e38)
        e = (z - high).exp()
        total = e.sum(-1, keepdim=True).clamp(min=1e-30)
        p, logp = e / total, torch.where(there, z - high - total.log(), 0.0)
    at = ids.clamp(min=0)
    loss = (p * (logp - logits.gather(1, at) + lse)).sum(-1)
    if not c["grad"]:
        return loss.to(x.dtype)
    live = there.any(-1, keepdim=True)
    q = (logits - lse).exp().scatter_add_(1, at, -p)
    dx = torch.matmul(q, w) * (live * s["dloss"][:, None] / tau)
    return [loss.to(x.dtype), dx.to(x.dtype)]


# --------------------------------------------------------------------------
def _handle(s):
    """The library's view of the weight and the adapters, made once as a user's program keeps them."""
    if "handle" not in s:
        import quantized_matvec_amd as qmv
        c = s["case"]
        s["qmv"] = qmv
        scales = {k: s[k] for k in ("absmax", "absmax_q", "absmax2", "offset", "code2") if k in s}
        s["handle"] = qmv.QuantState((s["rows"], c["K"]), s["x"].dtype, c["bs"], c["quant"], **scales)
        if "A" in s:
            s["adapters"] = qmv.LoraAdapters(s["A"], s["B"], s["scale"])
    return s["qmv"], s["handle"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_lora(s) if op.startswith("lora") else _plain_loss(s)
    qmv, state = _handle(s)
    if op == "lora":
        return qmv.lora_4bit(s["x"], s["packed"], state, s["adapters"], s["index"], bias=s["bias"])
    if op == "lora_backward":
        return qmv.lora_4bit_backward(s["dy"], s["x"], s["packed"], state, s["adapters"], s["index"])
    if op == "cross_entropy":
        return qmv.cross_entropy_4bit(s["x"], s["packed"], state, s["target"], dloss=s.get("dloss"))
    return qmv.distill_4bit(s["x"], s["packed"], state, s["ids"], s["teacher"], temperature=s["case"]["tau"], dloss=s.get("dloss"))


# --------------------------------------------------------------------------
# the definitions in 64 bits, adapter by adapter and in groups of tokens
# --------------------------------------------------------------------------
def _weight64(s, first, last):
    """Rows first .. last - 1 in float64."""
    c = s["case"]
    t = torch.tensor(NF4 if c["quant"] == "nf4" else FP4, device="cuda").double()
    K = c["K"]
    codes = s["packed"][first * K // 2:last * K // 2]
    w = torch.empty(last - first, K, dtype=torch.float64, device="cuda")
    w.view(-1)[0::2], w.view(-1)[1::2] = t[(codes // 16).long()], t[(codes % 16).long()]
    block = torch.arange(first * K // c["bs"], last * K // c["bs"], device="cuda")
    if c["double"]:  # the scale itself is defined with two fp32 roundings
        a = s["code2"][s["absmax_q"][block].long()] * s["absmax2"][block // 256]
        a = (a + s["offset"]).double()
    else:
        a = s["absmax"][block].double()
    return w.view(-1, c["bs"]).mul_(a[:, None]).view(last - first, K)


def exact(case, seed):
    s = prepare(case, seed)
    T = case["tokens"]
    x = s["x"].double()
    if case["op"].startswith("lora"):
        w = _weight64(s, 0, s["rows"])
        backward = case["op"] == "lora_backward"
        if backward:
            dy = s["dy"].double()
            dx, da, db = dy @ w, torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
        else:
            y = x @ w.t()
            if s["bias"] is not None:
                y += s["bias"].double()
        for a in range(case["n"]):
            mine = (s["index"] == a).nonzero()[:, 0]
            A, B, scale = s["A"][a].double(), s["B"][a].double(), s["scale"][a].double()
            if backward:
                v = scale * (dy[mine] @ B)
                dx[mine] += v @ A
                da[a], db[a] = v.t() @ x[mine], scale * dy[mine].t() @ (x[mine] @ A.t())
            else:
                y[mine] += scale * (x[mine] @ A.t() @ B.t())
        return [dx, da, db] if backward else y
    V, tau = s["rows"], case.get("tau", 1.0)
    w = _weight64(s, 0, V)
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    dx = torch.zeros(T, case["K"], dtype=torch.float64, device="cuda")
    for at in range(0, T, 512):
        rows = slice(at, min(T, at + 512))
        z = (x[rows] @ w.t()).div_(tau)
        logq = z.sub_(z.logsumexp(-1, keepdim=True))
        p = torch.zeros_like(logq)
        if case["op"] == "cross_entropy":
            live = s["target"][rows] >= 0
            t = torch.arange(len(live), device="cuda")[live]
            p[t, s["target"][rows][live]] = 1.0
        else:
            ids = s["ids"][rows]
            live = (ids >= 0).any(1)
            k = torch.where(ids >= 0, s["teacher"][rows].double() / tau, -torch.inf).softmax(-1)
            t, j = (ids >= 0).nonzero(as_tuple=True)
            p.index_put_((t, ids[t, j]), k[t, j], accumulate=True)
        loss[rows] = (torch.special.xlogy(p, p) - p * logq).sum(-1)
        if case["grad"]:
            dx[rows] = (logq.exp_() - p) @ w * (live * s["dloss"][rows].double() / tau)[:, None]
    return [loss, dx] if case["grad"] else loss
