"""The operators of include/qmv/tuning.h in 64 bits, token by token where that
says it plainest, and the error bounds derived for them.

Everything is float64 on the CPU over the fp32 dequantized weight W.  u is the
rounding of the activations' type (bounds.U), c32(n) = (n + 32) 2^-24 the fp32
roundings along any path of a sum of n terms.

Projection: |error| <= (u + c32(K)) sum |x||w| (the weight is rounded once, see
bounds.py).  The adapter's operands are taken as they are; its inner values
are fp32 sums carried in two 16-bit terms, off by at most T2 = u^2 of
themselves (2^-16, 2^-22) or by half of fp16's smallest number, 2^-25.  So its
part is off by at most (T2 + c32(inner) + c32(outer)) of the sum of the
magnitudes, plus 2^-25 sum |outer operand| in fp16.  One more rounding to the
output's type.

Loss: a logit is off by at most E_v = (u + c32(K)) sum |x||w| / tau, and
log sum exp is off by no more than the largest E_v.  exp, log and the
products around them are within 4 ulp of fp32 of values up to |l| in
magnitude: EXP(l) = 2^-21 (1 + |l|) covers the exponent's argument as well.
Gradient: each q_v is off by a factor within exp(+-2 E), the second product's
operands are rounded to 16 bits (u each; in fp16 terms below 2^-28 of the
largest are off by 2^-39 of it), its sum has V terms and one rescaling for
each piece.  A weight q_v that is below fp32's smallest normal number, 2^-126
(l_v is 87 below the largest), may be taken as 0 by exp, by a product or by the
matrix cores, which do not keep subnormals: up to 2^-126 |w_v| is lost there,
2^-126 sum |w| in all."""
from __future__ import annotations

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUB = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def c32(n):
    return (n + 32) * 2.0 ** -24


def _check(got, ref, bound, what):
    got = got.detach().double().cpu().reshape(ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - ref).abs()
    bad = (off > bound).nonzero()
    assert len(bad) == 0, (f"{what}: {len(bad)} of {ref.numel()} elements off by more than their bound, first {bad[:3].tolist()}: "
                           f"got {got[tuple(bad[0])]}, want {ref[tuple(bad[0])]}, bound {bound[tuple(bad[0])]}")


def _rounded(ref, bound, dtype):
    return 1.01 * (bound + U[dtype] * ref.abs() + SUB[dtype])


def check_lora(y, x, W, down, up, scale, index, bias=None, what="y"):
    """y against W x + bias + up (scale down x)."""
    dt, out = x.dtype, y.dtype
    x, W, down, up, scale, index = (t.detach().double().cpu() for t in (x, W, down, up, scale, index))
    T, (N, K) = x.shape[0], W.shape
    n, R = down.shape[:2]
    ref, mag = x @ W.T, x.abs() @ W.abs().T
    bound = (U[dt] + c32(K)) * mag + SUB[dt] * x.abs().sum(1, keepdim=True)
    for a in range(n):
        t = (index == a).nonzero()[:, 0]
        inner, minner = scale[a] * (x[t] @ down[a].T), scale[a].abs() * (x[t].abs() @ down[a].abs().T)
        ref[t] += inner @ up[a].T
        bound[t] += (U[dt] ** 2 + c32(K) + c32(2 * R)) * (minner @ up[a].abs().T)
        if dt == torch.float16:
            bound[t] += 2.0 ** -25 * up[a].abs().sum(1)
    if bias is not None:
        ref = ref + bias.double().cpu()
    _check(y, ref, _rounded(ref, bound + 2 * 2.0 ** -24 * ref.abs(), out), what)


def check_lora_backward(grads, dy, x, W, down, up, scale, index, what=""):
    dx, dd, du = grads
    dt, out = x.dtype, dd.dtype
    dy, x, W, down, up, scale, index = (t.detach().double().cpu() for t in (dy, x, W, down, up, scale, index))
    T, (N, K) = x.shape[0], W.shape
    n, R = down.shape[:2]
    sub = 2.0 ** -25 if dt == torch.float16 else 0.0
    ref, bound = dy @ W, (U[dt] + c32(N)) * (dy.abs() @ W.abs()) + SUB[dt] * dy.abs().sum(1, keepdim=True)
    for a in range(n):
        t = (index == a).nonzero()[:, 0]
        s = scale[a].abs()
        v, mv = scale[a] * (dy[t] @ up[a]), s * (dy[t].abs() @ up[a].abs())
        u, mu = scale[a] * (x[t] @ down[a].T), s * (x[t].abs() @ down[a].abs().T)
        ref[t] += v @ down[a]
        bound[t] += (U[dt] ** 2 + c32(N) + c32(2 * R)) * (mv @ down[a].abs()) + sub * down[a].abs().sum(0)
        r = v.T @ x[t]
        b = (U[dt] ** 2 + c32(N) + c32(2 * T)) * (mv.T @ x[t].abs()) + sub * x[t].abs().sum(0)
        _check(dd[a], r, _rounded(r, b, out), f"{what} d_down[{a}]")
        r = dy[t].T @ u
        b = (U[dt] ** 2 + c32(K) + c32(2 * T)) * (dy[t].abs().T @ mu) + sub * dy[t].abs().sum(0)[:, None]
        _check(du[a], r, _rounded(r, b, out), f"{what} d_up[{a}]")
    _check(dx, ref, _rounded(ref, bound + 2 * 2.0 ** -24 * ref.abs(), dt), f"{what} dx")


def target_p(ids, teacher, tau, V):
    """The target distribution over the vocabulary [T, V], and which tokens have one."""
    T, k = ids.shape
    there = (ids >= 0) & (ids < V)
    z = torch.where(there, torch.zeros(T, k).double() if teacher is None else teacher.detach().double().cpu() / tau, -torch.inf)
    live = (z > -torch.inf).any(1)
    p = torch.zeros(T, V, dtype=torch.float64)
    each = torch.zeros(T, k, dtype=torch.float64)
    for t in live.nonzero()[:, 0].tolist():
        each[t] = z[t].softmax(0)
        p[t].index_add_(0, ids[t][there[t]], each[t][there[t]])
    return p, each, live


def check_loss(loss, dx, x, W, ids, teacher=None, tau=1.0, dloss=None, exact_weights=False, what=""):
    """A loss (and dx) of rows x over the weight W; ids [T, k].  exact_weights:
    the weight's and logits' products are exact in the 16-bit type, E_v = 0."""
    dt, ldt = x.dtype, loss.dtype
    x, W, ids = x.detach().double().cpu(), W.detach().double().cpu(), ids.cpu()
    T, (V, K) = x.shape[0], W.shape
    p, each, live = target_p(ids, teacher, tau, V)
    l = x @ W.T / tau
    E = 0.0 if exact_weights else ((U[dt] + c32(K)) * (x.abs() @ W.abs().T) + SUB[dt] * x.abs().sum(1, keepdim=True)).amax(1) / tau
    lmax = l.abs().amax(1)
    E = E + 2.0 ** -21 * (1 + lmax)
    lse = l.logsumexp(1)
    there = (ids >= 0) & (ids < V)
    logq = (l - lse[:, None]).gather(1, ids.clamp(0, V - 1))
    terms = torch.special.xlogy(each, each) - torch.where(each > 0, each * logq, 0.0)
    ref = torch.where(live, terms.sum(1), 0.0)
    zabs = 0.0 if teacher is None else torch.where(there & torch.isfinite(teacher.cpu().double()), teacher.cpu().double().abs() / tau, 0.0).amax(1)
    bound = live * (2 * E + c32(V) + 2.0 ** -20 * (1 + zabs + ref.abs()))
    if teacher is None:  # near 0 the loss is log(1 + rest), not a difference
        rest = -torch.expm1(logq[:, 0].clamp(max=0.0))
        bound = torch.minimum(bound, live * (ref * (torch.expm1(2 * E) + c32(V) + 2.0 ** -20) + rest * 2.0 ** -20 + 2.0 ** -126)) \
            if exact_weights else bound
    _check(loss, ref, _rounded(ref, bound, ldt), f"{what} loss")
    if dx is None:
        return
    g = dloss.detach().double().cpu()[:, None] / tau * live[:, None]
    q = (l - lse[:, None]).exp()
    ref = g * ((q - p) @ W)
    # the ids' part is fp32 throughout: off by what q and p are
    hot = p > 0
    others = q * ~hot
    u = 0.0 if exact_weights else U[dt]
    spread = torch.expm1(2 * E)[:, None]
    b = (spread + U[dt] + u + c32(V) + 2.0 ** -20) * (others @ W.abs())
    zrel = 2.0 ** -20 * (1 + (zabs if teacher is not None else torch.zeros(T)))[:, None]
    one = (q * hot).sum(1, keepdim=True)
    if teacher is None:  # q - 1 comes from the others' sum
        b = b + ((spread + c32(V) + 2.0 ** -20) * (1 - one).clamp(min=0)) * (p @ W.abs()) * 1.0
    else:
        b = b + spread * ((q * hot) @ W.abs()) + zrel * (p @ W.abs()) + 2.0 ** -20 * ((q * hot) @ W.abs())
    if dt == torch.float16:
        top = torch.where(hot, -torch.inf, l - lse[:, None]).amax(1).exp()[:, None]
        b = b + 2.0 ** -39 * top * W.abs().sum(0)
    b = b + 2.0 ** -126 * W.abs().sum(0)
    b = g.abs() * (b + c32(ids.shape[1] + 64) * ((others + (q - p).abs()) @ W.abs()))
    _check(dx, ref, _rounded(ref, b, dt), f"{what} dx")
    assert (dx.cpu()[~live] == 0).all()
