"""Plain numpy forms in 64 bits of the 4-bit cache and of attention with a
window and sinks, and the error bounds their tests hold the kernels to.

Bounds of the decode (fp32 output), per output element.  With A = sum_j p_j
|v_j| over the visible tokens and B = scale * max_j sum_d |q_d k_jd|:
  * a score is an fp32 sum of 64 exact products: its error is below
    (64 + 16) * 2^-24 * B; exp2 adds 2^-21 relative; a relative error e of
    every weight moves the output by at most 2 e A (numerator, denominator);
  * the weights keep 22 bits (two fp16 halves) or 24 bits (three bf16 parts,
    2^-8 each time): e_p A, e_p = 2^-21 or 2^-23;
  * fp32 accumulation of n / 16 products, merges included: (n / 16 + 64) *
    2^-23 * A.
On the 4-bit cache a row enters as s (c - 7.5) + (z + 7.5 s) and its score as
s (q . c) + z sum(q), so |v| is at most 8 s + |z + 8 s| (7.5 s + |z + 7.5 s| is
no larger) and sum |q k| is (15 s + |z|) sum |q|.
"""
import numpy as np
import torch

D = 64
REC = 1152


def bf16_to_f64(bits):
    """uint16 bf16 bits -> float64."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16_bits(x):
    """float64 -> bf16 bits, round to nearest even (through torch)."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def unpack(cache):
    """uint8 [NB, bs/16, Hkv, 1152] -> codes [2, NB, bs, Hkv, 64] (K, V), s and
    z [2, NB, bs, Hkv] in float64."""
    nb, ch, hkv, _ = cache.shape
    codes, ss, zz = [], [], []
    for part in (0, 1):
        b = cache[..., 512 * part:512 * part + 512].reshape(nb, ch, hkv, 16, 32)
        c = np.stack([b & 15, b >> 4], axis=-1).reshape(nb, ch, hkv, 16, D)
        m = np.ascontiguousarray(cache[..., 1024 + 64 * part:1088 + 64 * part]).view(np.uint16)
        m = bf16_to_f64(m.reshape(nb, ch, hkv, 16, 2))
        codes.append(c.transpose(0, 1, 3, 2, 4).reshape(nb, ch * 16, hkv, D))
        ss.append(m[..., 0].transpose(0, 1, 3, 2).reshape(nb, ch * 16, hkv))
        zz.append(m[..., 1].transpose(0, 1, 3, 2).reshape(nb, ch * 16, hkv))
    return np.stack(codes), np.stack(ss), np.stack(zz)


def values(cache):
    c, s, z = unpack(cache)
    return c * s[..., None] + z[..., None]


def quantise(rows):
    """Rows [..., 64] (float64 holding bf16 numbers) -> codes, s, z by the
    definition, in 64 bits (s rounded up to 8 significant bits)."""
    z = rows.min(-1)
    m, e = np.frexp((rows.max(-1) - z) / 15.0)
    s = np.ldexp(np.ceil(m * 256.0), e - 8)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.rint((rows - z[..., None]) / s[..., None]), 0.0)
    return np.clip(c, 0, 15).astype(np.uint8), s, z


def random_cache(rng, nb, bs, hkv, spread=1.0):
    """A 4-bit cache of quantised normal rows (every slot used)."""
    cache = np.zeros((nb, bs // 16, hkv, REC), np.uint8)
    for part in (0, 1):
        x = bf16_to_f64(f64_to_bf16_bits(rng.standard_normal((nb, bs // 16, hkv, 16, D)) * spread))
        c, s, z = quantise(x)
        cache[..., 512 * part:512 * part + 512] = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(nb, bs // 16, hkv, 512)
        sz = np.stack([f64_to_bf16_bits(s), f64_to_bf16_bits(z)], axis=-1)
        cache[..., 1024 + 64 * part:1088 + 64 * part] = np.ascontiguousarray(sz).view(np.uint8).reshape(nb, bs // 16, hkv, 64)
    return cache


def visible(pos, window, sinks):
    """Visible token positions of a query at `pos`."""
    j = np.arange(pos + 1)
    return j if window == 0 else j[(j > pos - window) | (j < sinks)]


def attend(q, k, v, scale, absq=None, absv=None):
    """One query row over rows k, v [n, 64]: output, A (see above), B."""
    s = k @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    av = np.abs(v) if absv is None else absv
    b = (np.abs(k) @ np.abs(q) if absq is None else absq * np.abs(q).sum()).max() * abs(scale)
    return p @ v, p @ av, abs(b)


def decode_bound(a, b, n, split_bits):
    return a * (2 * (80 * 2.0 ** -24 * b + 2.0 ** -21) + 2.0 ** -split_bits + (n / 16 + 64) * 2.0 ** -23) + 1e-37


def decode_ref(q, tables, ctx, scale, window, sinks, kv=None, cache=None):
    """fp64 decode and its error bound: q [S, Hq, 64]; kv = (K, V) [NB, bs,
    Hkv, 64] in float64, or the 4-bit cache."""
    s_n, hq, _ = q.shape
    if cache is not None:
        codes, ss, zz = unpack(cache)
        K, V = (codes[i] * ss[i][..., None] + zz[i][..., None] for i in (0, 1))
    else:
        K, V = kv
    bs, hkv = K.shape[1], K.shape[2]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for s in range(s_n):
        if ctx[s] <= 0:
            continue
        pos = visible(int(ctx[s]) - 1, window, sinks)
        page, off = tables[s][pos // bs], pos % bs
        for h in range(hq):
            g = h // (hq // hkv)
            k, v = K[page, off, g], V[page, off, g]
            absq = absv = None
            if cache is not None:
                absq = 15 * ss[0][page, off, g] + np.abs(zz[0][page, off, g])
                sv = ss[1][page, off, g]
                absv = np.repeat((8 * sv + np.abs(zz[1][page, off, g] + 8 * sv))[:, None], D, 1)
            o, a, b = attend(q[s, h], k, v, scale, absq, absv)
            out[s, h] = o
            tol[s, h] = decode_bound(a, b, len(pos), 21 if cache is not None else 23)
    return out, tol


def deal(rng, ctx, bs, extra=3):
    """Scattered block tables for contexts `ctx`; returns (tables, NB)."""
    nblk = [-(-int(c) // bs) for c in ctx]
    nb = sum(nblk) + extra
    perm = rng.permutation(nb).astype(np.int32)
    mb = max(1, max(nblk))
    tables = np.full((len(ctx), mb), -1, np.int32)
    at = 0
    for s, n in enumerate(nblk):
        tables[s, :n] = perm[at:at + n]
        at += n
    return tables, nb


def bf16(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).to(dev)


def f64(t):
    return t.detach().double().cpu().numpy()
