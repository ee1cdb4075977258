"""Plain numpy form in 64 bits of differential attention, and the error bound its
tests hold the kernels to.

The bf16 output is rounded once, 2^-8 of itself.  Before that, for each map with
A = sum_j p_j |v_j| and B = scale * max_j sum_d |q_d k_jd| (as in window_common):
  e = A * (2 * (80 * 2^-24 * B + 2^-21) + 2^-bits + (n / 16 + 64) * 2^-23)
with the weights kept in `bits` bits: 2^-15 in the decode (two bf16 parts, 2^-8 each
time, with one bit to spare), 2^-11 in the prefill (fp16), whose P.V also adds n / 8
products in the tensor core: (n / 8 + 64) * 2^-23, V below 2^-14 keeps an absolute
error of 2^-25, and so does a weight below 2^-14 of the reference's (whose sum is at
least 1): 2^-25 sum_j |v_j|.  d = o1 - lambda o2 is then off by E = e1 + |lambda| e2 +
2^-22 (|o1| + |lambda o2|).  The norm divides by r = sqrt(mean d^2 + eps):
  |error of d_i / r| <= E_i / r + |d_i| / r * (rms(E) / r + 2^-21),
where r is taken as at least r - rms(E) in the denominators.
"""
import numpy as np

import window_common as C

DV = 128


def attend(q, k, v, scale, bits, prefill):
    """One map of one query row: output and its error bound, [128] each."""
    o, a, b = C.attend(q, k, v, scale)
    n = len(k)
    e = a * (2 * (80 * 2.0 ** -24 * b + 2.0 ** -21) + 2.0 ** -bits + (n / (8 if prefill else 16) + 64) * 2.0 ** -23)
    return o, e + (2.0 ** -25 * (1 + np.abs(v).sum(0)) if prefill else 1e-37)


def pair_row(q1, q2, k1, k2, v, scale, lam, weight, eps, out_scale, bits, prefill=False):
    """One row of one query pair: value and bound, the bf16 rounding included."""
    o1, e1 = attend(q1, k1, v, scale, bits, prefill)
    o2, e2 = attend(q2, k2, v, scale, bits, prefill)
    d = o1 - lam * o2
    err = e1 + abs(lam) * e2 + 2.0 ** -22 * (np.abs(o1) + np.abs(lam * o2))
    if weight is None:
        y, tol = d * out_scale, err * abs(out_scale)
    else:
        r = np.sqrt(np.mean(d * d) + eps)
        y = np.zeros_like(d) if r == 0 else out_scale * weight * d / r
        slip = np.sqrt(np.mean(err * err))
        low = max(r - slip, np.sqrt(eps), 1e-300)
        tol = np.abs(out_scale * weight) / low * (err + np.abs(d) * (slip / low + 2.0 ** -21))
    return y, tol + (np.abs(y) + tol) * 2.0 ** -8


def reference(q, starts, tables, ctx, k, v, lam, scale, window=0, sinks=0, weight=None, eps=1e-5,
              out_scale=1.0, bits=15, prefill=False):
    """q [T, Hq, 64]; rows starts[s] .. starts[s + 1] are the last of sequence s; k, v
    [NB, bs, Hkv, 64] in float64; lam [pairs] or [T, pairs].  Values and bounds [T, pairs, 128]."""
    t, hq, _ = q.shape
    bs, hkv = k.shape[1], k.shape[2]
    g = hq // hkv
    lam = np.broadcast_to(lam, (t, hq // 2))
    out, tol = np.zeros((t, hq // 2, DV)), np.zeros((t, hq // 2, DV))
    for s, n in enumerate(ctx):
        rows = starts[s + 1] - starts[s]
        for i in range(rows):
            pos = C.visible(int(n) - rows + i, window, sinks)
            if n <= 0:
                continue
            page, off = tables[s][pos // bs], pos % bs
            r = starts[s] + i
            for p in range(hq // 2):
                j = p // g
                kk = k[page, off][:, 2 * j:2 * j + 2]
                vv = v[page, off, 2 * j:2 * j + 2].reshape(len(pos), DV)
                out[r, p], tol[r, p] = pair_row(q[r, 2 * p], q[r, 2 * p + 1], kk[:, 0], kk[:, 1], vv, scale,
                                                lam[r, p], weight, eps, out_scale, bits, prefill)
    return out, tol
