"""Plain float64 forms of the rotary, cache and attention operators (numpy, on
the CPU), and the error bounds that their tests hold the kernels to.

Attention's bound, to first order.  With s_j the scores and p_j the softmax
weights of a row, a kernel may differ from out = sum p_j v_j by
* the rounding of the code values to fp16 (11 significant bits, 2^-11) in the
  keys, and of the queries, which keep 11 bits below the row's largest
  magnitude times 2^-14: score j is off by at most
      e_j = |scale| ((2^-11 + (D + 16) 2^-24) sum |q_d k_jd| + D 2^-25 max|q| max|k_j|)
            + 2^-21 (|s_j| + max |s|)      (fp32 scaling, exponent argument, exp2)
  which moves weight j by e_j relatively and their sum by sum p_j e_j;
* the same rounding of the values' code values, and of the weights times the
  block scale to fp16: 2 2^-11 relative, and 2^-38 of the largest
  such product absolutely;
* fp32 sums over the L keys of a row, their partial results and the rescaling
  of the running sums: (L + 64) 2^-24;
* the one rounding of the output to its type.
Per element:
    |out - ref| <= sum_j p_j |v_jd| (e_j + e + 2 2^-11 + (L + 64) 2^-23)
                   + L 2^-38 max|v| + u_out |ref| + subnormal term, e = sum p_j e_j
"""
import numpy as np

import oracle as O

U_OUT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
SUBNORMAL = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}


def rope_frequencies(rot, theta):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def rope_table(freqs, max_pos, gain=1.0):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * np.asarray(freqs, np.float64)
    return np.stack([gain * np.cos(a), gain * np.sin(a)], -1).astype(np.float32)


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, table, positions, interleaved, inverse=False, dtype=np.float64):
    """x [T, H, D] turned; with dtype float32 every product and sum rounds as
    the kernels' do."""
    x = np.asarray(x, dtype)
    out = x.copy()
    rot = 2 * table.shape[1]
    ia, ib = pairs(rot, interleaved)
    for t, p in enumerate(positions):
        if not 0 <= p < table.shape[0]:
            out[t] = 0
            continue
        c, s = table[p, :, 0].astype(dtype), table[p, :, 1].astype(dtype)
        if inverse:
            s = -s
        a, b = x[t][:, ia], x[t][:, ib]
        out[t][:, ia] = a * c - b * s
        out[t][:, ib] = b * c + a * s
    return out


def encode_rows(x, bs, qt):
    """Packed codes [..., D / 2] and block maxima [..., D / bs] by the codec's oracle."""
    x = np.asarray(x, np.float64)
    p, a = O.quantize_4bit(x.reshape(-1), bs, qt)
    return p.reshape(x.shape[:-1] + (x.shape[-1] // 2,)), np.asarray(a, np.float64).reshape(x.shape[:-1] + (-1,))


def decode_rows(codes, scales, qt):
    t = O.code_table(qt).astype(np.float64)
    dim = 2 * codes.shape[-1]
    x = np.stack([t[codes >> 4], t[codes & 15]], -1).reshape(scales.shape + (dim // scales.shape[-1],))
    return (x * scales[..., None]).reshape(codes.shape[:-1] + (dim,))


def attend(q, k, v, scale, lo, hi):
    """One sequence and cache head: q [R, D], k and v [L, D], row r seeing keys
    lo[r] <= j < hi[r] of those marked there.  Returns (out, bound without the
    output's rounding)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    R, D = q.shape
    out, bound = np.zeros((R, D)), np.zeros((R, D))
    for r in range(R):
        j = np.arange(max(lo[r], 0), max(hi[r], 0))
        j = j[~np.isnan(k[j, 0])]          # keys of pages that are not there are NaN rows
        if j.size == 0:
            continue
        kk, vv = k[j], v[j]
        s = scale * (kk @ q[r])
        p = np.exp(s - s.max())
        p /= p.sum()
        out[r] = p @ vv
        L = j.size
        e = abs(scale) * ((2.0 ** -11 + (D + 16) * 2.0 ** -24) * (np.abs(kk) @ np.abs(q[r]))
                          + D * 2.0 ** -25 * np.abs(q[r]).max() * np.abs(kk).max(1)) \
            + 2.0 ** -21 * (np.abs(s) + np.abs(s).max())
        rel = e + (p * e).sum() + 2 * 2.0 ** -11 + (L + 64) * 2.0 ** -23
        bound[r] = (p * rel) @ np.abs(vv) + L * 2.0 ** -38 * np.abs(vv).max()
    return out, bound
