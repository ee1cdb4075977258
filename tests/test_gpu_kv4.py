"""The 4-bit cache on the GPU: the quantising write (with and without the
rotary embedding), expansion, block copies and the decode attention, against
plain forms in 64 bits (tests/window_common.py, which also derives the decode's
bounds)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_198_gb300 as tvl
import window_common as C
from gpu_common import DEV, assert_clean_status

pytestmark = pytest.mark.gpu


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


# --------------------------------------------------------------------- write


@pytest.mark.parametrize("bs,hkv,t", [(16, 8, 300), (32, 1, 1), (64, 3, 77), (128, 12, 130), (16, 9, 33)])
def test_write_is_the_definition(bs, hkv, t):
    """Without rotation every code, s and z equals the 64-bit definition's: x -
    z, the quotients and the ties are exact in fp32 for bf16 rows of like
    magnitude.  Slots that are not written keep their bytes."""
    rng = np.random.default_rng(10 + t)
    nb = t // bs + 3
    before = C.random_cache(rng, nb, bs, hkv)
    scale = 2.0 ** rng.integers(-6, 5, (t, hkv, 1))
    k, v = (C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((t, hkv, 64)) * scale)) for _ in range(2))
    k[0, 0] = 0.75                                   # a constant row: s = 0
    v[-1, -1, :32] = 0.0
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    slots[t // 2::7] = -1
    cache = _cuda(before)
    tvl.kv4_write(C.bf16(k, DEV), C.bf16(v, DEV), cache, _cuda(slots))
    got, s, z = C.unpack(cache.cpu().numpy())
    want, s0, z0 = C.unpack(before)
    live = slots >= 0
    page, off = slots[live] // bs, slots[live] % bs
    for part, x in ((0, k), (1, v)):
        c, ss, zz = C.quantise(x[live])
        want[part][page, off], s0[part][page, off], z0[part][page, off] = c, ss, zz
    assert np.array_equal(s, s0) and np.array_equal(z, z0)
    assert np.array_equal(got, want)
    assert_clean_status()


@pytest.mark.parametrize("theta,with_q", [(500000.0, True), (10000.0, True), (10000.0, False)])
def test_write_with_rope(theta, with_q):
    """q and K against the double-precision rotation: one bf16 ulp (2^-7 of
    the value) plus 2^-21 of the pair for q, and for K half a step more."""
    rng = np.random.default_rng(3)
    t, hq, hkv, bs, nb = 200, 24, 4, 32, 9
    q, k, v = (C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((t, h, 64)))) for h in (hq, hkv, hkv))
    pos = rng.integers(0, 200000, t).astype(np.int32)
    pos[:4] = [0, 1, 2 ** 31 - 1, 131071]
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    slots[5] = -1
    ang = pos[:, None].astype(np.float64) * float(np.float32(theta)) ** (-2.0 * np.arange(32) / 64)
    cos, sin = np.cos(ang)[:, None], np.sin(ang)[:, None]

    def rot(x):
        a, b = x[..., :32], x[..., 32:]
        return np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)

    def room(x, y):
        pair = np.abs(x[..., :32]) + np.abs(x[..., 32:])
        # far positions: the reduced angle itself is good to 2^-52 of the full one
        return np.abs(y) * 2.0 ** -7 + np.concatenate([pair, pair], -1) * (2.0 ** -21 + ang.max() * 2.0 ** -50)

    cache = torch.zeros(tvl.kv4_cache_shape(nb, hkv, bs), dtype=torch.uint8, device=DEV)
    dq = C.bf16(q, DEV) if with_q else None
    tvl.kv4_write(C.bf16(k, DEV), C.bf16(v, DEV), cache, _cuda(slots), q=dq, positions=_cuda(pos),
                  rope_theta=theta)
    if with_q:
        y = rot(q)
        assert (np.abs(C.f64(dq) - y) <= room(q, y)).all()
    val = C.values(cache.cpu().numpy())
    codes, s, z = C.unpack(cache.cpu().numpy())
    live = slots >= 0
    page, off = slots[live] // bs, slots[live] % bs
    y = rot(k)[live]
    step = s[0][page, off][..., None]
    assert (np.abs(val[0][page, off] - y) <= room(k, rot(k))[live] + step * (0.5 + 2.0 ** -20)).all()
    c, ss, zz = C.quantise(v[live])
    assert np.array_equal(codes[1][page, off], c) and np.array_equal(z[1][page, off], zz)
    assert_clean_status()


def test_write_reports_bad_slots_and_rows():
    rng = np.random.default_rng(4)
    before = C.random_cache(rng, 2, 16, 2)
    cache = _cuda(before)
    k = rng.standard_normal((4, 2, 64))
    k[1, 0, 7] = np.nan
    k[2, 1, 63] = np.inf
    tvl.kv4_write(C.bf16(k, DEV), C.bf16(np.ones((4, 2, 64)), DEV), cache,
                  _cuda(np.array([3, 9, 31, 32], np.int32)))
    assert tvl.get_device_status() == tvl.DEV_BAD_SLOT | tvl.DEV_NONFINITE
    val = C.values(cache.cpu().numpy())
    assert np.isnan(val[0][0, 9, 0]).all() and np.isnan(val[0][1, 15, 1]).all()
    assert np.isfinite(val[0][0, 9, 1]).all() and np.isfinite(val[0][0, 3]).all()
    old = C.values(before)
    for part in (0, 1):                              # every other slot as it was
        keep = np.ones((2, 16), bool)
        keep[0, 3] = keep[0, 9] = keep[1, 15] = False
        assert np.array_equal(val[part][keep], old[part][keep])


def test_write_of_nothing_and_of_padding_only():
    cache = torch.zeros(tvl.kv4_cache_shape(2, 2, 16), dtype=torch.uint8, device=DEV)
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    tvl.kv4_write(e, e, cache, torch.zeros(0, dtype=torch.int32, device=DEV))
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    tvl.kv4_write(k, k, cache, torch.full((3,), -1, dtype=torch.int32, device=DEV))
    assert int(cache.sum()) == 0
    assert_clean_status()


# ------------------------------------------------------------ expand and copy


@pytest.mark.parametrize("bs,hkv", [(16, 8), (128, 3), (32, 1)])
def test_expand_rounds_the_value_once(bs, hkv):
    """bf16(s c + z): the product is exact in fp32 (4 by 8 bits), the sum is
    rounded to 24 bits and then to 8, so off by half a bf16 step and 2^-24."""
    rng = np.random.default_rng(5)
    cache = C.random_cache(rng, 6, bs, hkv)
    kc = torch.full((9, bs, hkv, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    src, dst = np.array([4, 0, 5], np.int32), np.array([8, 2, 0], np.int32)
    tvl.kv4_expand_blocks(kc, vc, _cuda(cache), _cuda(src), _cuda(dst))
    val = C.values(cache)
    for part, got in ((0, C.f64(kc)), (1, C.f64(vc))):
        want = val[part][src]
        assert (np.abs(got[dst] - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -24 * 16).all()
        rest = np.setdiff1d(np.arange(9), dst)
        assert (got[rest] == 7.0).all()
    assert_clean_status()


def test_expand_and_copy_report_bad_blocks():
    rng = np.random.default_rng(6)
    before = C.random_cache(rng, 4, 16, 2)
    cache = _cuda(before)
    tvl.kv4_copy_blocks(cache, _cuda(np.array([0, 9, 1], np.int32)), _cuda(np.array([3, 2, -1], np.int32)))
    assert tvl.get_device_status() == tvl.DEV_BAD_BLOCK_ID
    want = before.copy()
    want[3] = before[0]
    assert np.array_equal(cache.cpu().numpy(), want)
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    tvl.kv4_expand_blocks(kc, kc.clone(), cache, _cuda(np.array([0, 4], np.int32)),
                          _cuda(np.array([2, 0], np.int32)))
    assert tvl.get_device_status() == tvl.DEV_BAD_BLOCK_ID
    assert float(kc.float().abs().sum()) == 0.0


@pytest.mark.parametrize("bs,hkv", [(16, 8), (64, 5)])
def test_copy_is_bit_exact(bs, hkv):
    rng = np.random.default_rng(7)
    before = C.random_cache(rng, 5, bs, hkv)
    cache = _cuda(before)
    tvl.kv4_copy_blocks(cache, _cuda(np.array([4, 0], np.int32)), _cuda(np.array([1, 3], np.int32)))
    want = before.copy()
    want[1], want[3] = before[4], before[0]
    assert np.array_equal(cache.cpu().numpy(), want)


# -------------------------------------------------------------------- decode


def _decode(seed, ctx, hq, hkv, bs, window=0, sinks=0, spread=1.0, qscale=1.5, cache=None, scale=0.125):
    rng = np.random.default_rng(seed)
    tables, nb = C.deal(rng, ctx, bs)
    if cache is None:
        cache = C.random_cache(rng, nb, bs, hkv, spread)
    q = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((len(ctx), hq, 64)) * qscale))
    out = torch.full((len(ctx), hq, 64), float("nan"), device=DEV)
    tvl.kv4_attention_decode(out, C.bf16(q, DEV), _cuda(cache), _cuda(tables),
                             _cuda(np.asarray(ctx, np.int32)), scale, window=window, sinks=sinks)
    want, tol = C.decode_ref(q, tables, ctx, scale, window, sinks, cache=cache)
    return C.f64(out), want, tol


@pytest.mark.parametrize("hq,hkv,bs", [
    (8, 2, 16), (32, 8, 16), (8, 8, 32), (64, 8, 32), (5, 5, 64), (6, 1, 128), (21, 3, 16),
    (24, 12, 32), (14, 7, 16), (16, 16, 64), (8, 1, 16), (40, 8, 16)])
def test_decode_heads(hq, hkv, bs):
    got, want, tol = _decode(20 + hq, [1, 700, 16, 17, 333], hq, hkv, bs)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    assert_clean_status()


@pytest.mark.parametrize("ctx", [[1], [15], [16], [31, 33], [0, 5, 0], [0], [2000], [64] * 40,
                                 list(range(1, 200, 3))])
def test_decode_lengths(ctx):
    got, want, tol = _decode(40, ctx, 8, 2, 16)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert_clean_status()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (100, 16), (100, 17),
                                          (64, 1000), (5000, 4), (640, 300)])
@pytest.mark.parametrize("bs", [16, 64])
def test_decode_window(window, sinks, bs):
    got, want, tol = _decode(50, [1, 90, 101, 1500, 640, 116], 12, 3, bs, window, sinks)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    assert_clean_status()


@pytest.mark.parametrize("spread,qscale", [(1e-6, 1.0), (1e6, 1e-6), (0.01, 300.0), (30.0, 1e-3)])
def test_decode_magnitudes(spread, qscale):
    """Rows and queries far from 1: the powers of two folded into q and V."""
    got, want, tol = _decode(60, [500, 77], 16, 4, 16, spread=spread, qscale=qscale)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
@pytest.mark.parametrize("hq", [8, 16])
def test_decode_scales(scale, hq):
    got, want, tol = _decode(59, [100, 333], hq, 2, 16, 70, 3, scale=scale, qscale=0.3)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


def test_decode_of_constant_rows():
    """V rows of one value each (s = 0), so every weight meets a zero scale."""
    rng = np.random.default_rng(58)
    ctx = [50, 400]
    tables, nb = C.deal(np.random.default_rng(57), ctx, 16)
    cache = C.random_cache(rng, nb, 16, 2)
    cache[..., 512:1024] = 0
    meta = cache[..., 1088:1152].view(np.uint16).reshape(nb, 1, 2, 16, 2)
    meta[..., 0] = 0
    got, want, tol = _decode(57, ctx, 8, 2, 16, cache=cache)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


def test_decode_mixed_value_scales():
    """V rows whose scales differ by 2^40 within one context."""
    rng = np.random.default_rng(8)
    ctx, bs, hkv = [300, 40], 16, 2
    tables, nb = C.deal(np.random.default_rng(61), ctx, bs)
    cache = C.random_cache(rng, nb, bs, hkv)
    meta = cache[..., 1088:1152].view(np.uint16).reshape(nb, 1, hkv, 16, 2)
    e = rng.integers(-20, 21, (nb, 1, hkv, 16, 1)).astype(np.int32) << 7
    meta[...] = (meta.astype(np.int32) + e).astype(np.uint16)      # bf16 exponents moved together
    cache[..., 1088:1152] = np.ascontiguousarray(meta).view(np.uint8).reshape(nb, 1, hkv, 64)
    got, want, tol = _decode(61, ctx, 8, hkv, bs, cache=cache)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


def test_decode_ignores_unseen_slots():
    """NaN rows past the context, before the window and behind the last
    sequence, in blocks that are read, change nothing."""
    ctx, bs, hkv = [100, 333], 32, 2
    window, sinks = 50, 3
    got0, want, tol = _decode(62, ctx, 8, hkv, bs, window, sinks)
    rng = np.random.default_rng(62)
    tables, nb = C.deal(rng, ctx, bs)
    cache = C.random_cache(rng, nb, bs, hkv)
    seen = np.zeros((nb, bs), bool)
    for s, n in enumerate(ctx):
        p = C.visible(n - 1, window, sinks)
        seen[tables[s][p // bs], p % bs] = True
    for b in range(nb):
        for o in range(bs):
            if not seen[b, o]:
                for base in (1024, 1088):
                    cache[b, o // 16, :, base + 4 * (o % 16):base + 4 * (o % 16) + 4] = 0xff   # NaN
    got, _, _ = _decode(62, ctx, 8, hkv, bs, window, sinks, cache=cache)
    # _decode draws the cache before q: draw it here too, so that q is the same
    rng2 = np.random.default_rng(62)
    C.deal(rng2, ctx, bs)
    assert np.isfinite(got).all()
    want2, tol2 = _redo(rng2, cache, tables, ctx, window, sinks)
    assert (np.abs(got - want2) <= tol2).all()


def _redo(rng, cache, tables, ctx, window, sinks):
    q = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((len(ctx), 8, 64)) * 1.5))
    clean = cache.copy()
    return C.decode_ref(q, tables, ctx, 0.125, window, sinks, cache=clean)


def test_decode_of_a_nan_row_is_nan_for_its_head_alone():
    ctx, bs, hkv = [40], 16, 2
    rng = np.random.default_rng(63)
    tables, nb = C.deal(rng, ctx, bs)
    cache = C.random_cache(rng, nb, bs, hkv)
    b = tables[0][1]
    cache[b, 0, 1, 1024 + 4 * 3:1024 + 4 * 3 + 4] = 0xff          # K of token 19, head 1
    got, want, tol = _decode(63, ctx, 8, hkv, bs, cache=cache)
    assert np.isnan(got[0, 4:]).all()
    assert (np.abs(got - want) <= tol)[0, :4].all()


def test_decode_reports_bad_tables_and_lengths():
    rng = np.random.default_rng(64)
    cache = _cuda(C.random_cache(rng, 8, 16, 2))
    q = C.bf16(rng.standard_normal((2, 4, 64)), DEV)
    out = torch.zeros(2, 4, 64, device=DEV)
    tables = np.array([[0, 1, 99], [2, 3, 4]], np.int32)
    tvl.kv4_attention_decode(out, q, cache, _cuda(tables), _cuda(np.array([48, 48], np.int32)), 0.125)
    assert tvl.get_device_status() == tvl.DEV_BAD_BLOCK_ID
    tables[0, 2] = 5
    tvl.kv4_attention_decode(out, q, cache, _cuda(tables), _cuda(np.array([-3, 4000], np.int32)), 0.125)
    assert tvl.get_device_status() == tvl.DEV_BAD_CONTEXT_LEN
    assert float(out[0].abs().sum()) == 0.0


def test_decode_repeats_bit_for_bit_and_leaves_the_batch_alone():
    """Same call twice, on another stream, and from a captured graph."""
    rng = np.random.default_rng(65)
    ctx = [3, 900, 0, 450, 77]
    tables, nb = C.deal(rng, ctx, 16)
    cache, tab, ln = _cuda(C.random_cache(rng, nb, 16, 8)), _cuda(tables), _cuda(np.asarray(ctx, np.int32))
    q = C.bf16(rng.standard_normal((5, 32, 64)), DEV)
    outs = [torch.full((5, 32, 64), float("nan"), device=DEV) for _ in range(3)]
    tvl.kv4_attention_decode(outs[0], q, cache, tab, ln, 0.125)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tvl.kv4_attention_decode(outs[1], q, cache, tab, ln, 0.125)
        call = tvl.bind_kv4_attention_decode(outs[2], q, cache, tab, ln, 0.125)
        call()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(tvl.window_decode_workspace_size(32, 8), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(g):
        tvl.kv4_attention_decode(outs[1], q, cache, tab, ln, 0.125, workspace=ws)
    for _ in range(2):
        outs[1].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    assert_clean_status()


def test_workspace_too_small_is_refused():
    rng = np.random.default_rng(66)
    cache = _cuda(C.random_cache(rng, 4, 16, 2))
    q = C.bf16(rng.standard_normal((1, 4, 64)), DEV)
    out = torch.zeros(1, 4, 64, device=DEV)
    need = tvl.window_decode_workspace_size(4, 2)
    with pytest.raises(tvl.TvlError) as e:
        tvl.kv4_attention_decode(out, q, cache, _cuda(np.zeros((1, 2), np.int32)),
                                 _cuda(np.array([20], np.int32)), 0.125,
                                 workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == tvl.ERR_WORKSPACE


# ------------------------------------------------------------- used together


def test_serving_run_on_a_4bit_cache():
    """Prompt written with rotation, a fork with copy-on-write, a few decode
    steps: after each the attention equals the plain form over what the cache
    holds, and the rows it holds are the written ones within half a step."""
    rng = np.random.default_rng(67)
    hq, hkv, bs, nb = 8, 2, 16, 24
    alloc = tvl.BlockAllocator(nb, bs)
    cache = torch.zeros(tvl.kv4_cache_shape(nb, hkv, bs), dtype=torch.uint8, device=DEV)
    a = alloc.new_sequence()

    def append(seqs, n):
        at = np.concatenate([np.arange(alloc.context_len(s), alloc.context_len(s) + n) for s in seqs])
        slots = np.concatenate([alloc.append(s, n) for s in seqs])
        src, dst = alloc.take_copies()
        if len(src):
            tvl.kv4_copy_blocks(cache, _cuda(src), _cuda(dst))
        t = len(slots)
        k, v, q = (C.bf16(rng.standard_normal((t, h, 64)), DEV) for h in (hkv, hkv, hq))
        tvl.kv4_write(k, v, cache, _cuda(slots), q=q, positions=_cuda(at.astype(np.int32)))
        return q

    append([a], 37)
    b = alloc.fork(a)
    for step in range(12):
        q = append([a, b], 1)
        tables, ctx = alloc.build_tables([a, b], 8)
        out = torch.empty(2, hq, 64, device=DEV)
        tvl.kv4_attention_decode(out, q, cache, _cuda(tables), _cuda(ctx), 0.125)
        want, tol = C.decode_ref(C.f64(q), tables, ctx, 0.125, 0, 0, cache=cache.cpu().numpy())
        assert (np.abs(C.f64(out) - want) <= tol).all(), step
    assert alloc.stats()["shared_blocks"] == 2
    assert_clean_status()


@pytest.mark.parametrize("group", range(1, 9))
@pytest.mark.parametrize("ctx,window,sinks", [(2048, 0, 0), (2047, 0, 0), (4000, 1900, 90), (4000, 2016, 0)])
def test_decode_the_longest_sequences_of_few(group, ctx, window, sinks):
    """Few short bounded sequences: around the most chunks that one CTA holds."""
    got, want, tol = _decode(90 + group, [ctx, 40], group, 1, 16, window, sinks)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert_clean_status()


def _put(cache, tables, bs, pos, part, code, s, z):
    """Sets rows of the 4-bit cache, all heads: at positions pos of sequence 0, K
    (part 0) or V rows of codes `code` (a number or 64), scales s and minima z."""
    nib = np.broadcast_to(np.asarray(code, np.uint8), (64,))
    packed = nib[0::2] | nib[1::2] << 4
    for i, p in enumerate(pos):
        block, sub, tok = tables[0][p // bs], p % bs // 16, p % 16
        cache[block, sub, :, 512 * part + 32 * tok:512 * part + 32 * tok + 32] = packed
        sz = C.f64_to_bf16_bits(np.array([np.broadcast_to(s, len(pos))[i], np.broadcast_to(z, len(pos))[i]]))
        cache[block, sub, :, 1024 + 64 * part + 4 * tok:1028 + 64 * part + 4 * tok] = sz.view(np.uint8)


def _planned(n, hq, hkv, logits, v, window=0, bs=16):
    """One sequence of n tokens whose scores are `logits` (natural units; exact: K
    rows of one value, q of one 8) and whose V rows are v = (codes, s, z), each a
    number or one a token.  Returns the output, the plain form's and A = sum p
    (8 s + |z + 8 s|) of the bounds."""
    rng = np.random.default_rng(n)
    tables, nb = C.deal(rng, [n], bs)
    cache = np.zeros(tvl.kv4_cache_shape(nb, hkv, bs), np.uint8)
    _put(cache, tables, bs, range(n), 0, 0, 0.0, logits)
    _put(cache, tables, bs, range(n), 1, v[0], v[1], v[2])
    q = np.zeros((1, hq, 64))
    q[..., 5] = 8.0
    out = torch.full((1, hq, 64), float("nan"), device=DEV)
    tvl.kv4_attention_decode(out, C.bf16(q, DEV), _cuda(cache), _cuda(tables), _cuda(np.array([n], np.int32)),
                             0.125, window=window)
    _, _, z = C.unpack(cache)
    pos = C.visible(n - 1, window, 0)
    page, off = tables[0][pos // bs], pos % bs
    x = z[0][page, off, 0]
    p = np.exp(x - x.max())
    p /= p.sum()
    codes, s, z = (y[1][page, off, 0] for y in C.unpack(cache))
    a = (p * (8 * s + np.abs(z + 8 * s))).sum()
    spread = float(np.ptp(np.where(p > 0, x, x.max()))) / np.log(2.0)
    return C.f64(out)[0], p @ (codes * s[:, None] + z[:, None]), a, spread


def _planned_bound(n, a, spread):
    """decode_bound with scores that are exact but for the product with log2 e
    (and the reference's subtraction in one rounding): 2 * 2^-24 of their range."""
    return a * (2 * (2 * 2.0 ** -24 * spread + 2.0 ** -21) + 2.0 ** -21 + (n / 16 + 64) * 2.0 ** -23) + 1e-37


@pytest.mark.parametrize("hq,hkv", [(2, 1), (8, 1), (128, 32), (256, 32)])
@pytest.mark.parametrize("value", [2.0 ** 59, -100.0, 2.0 ** -80, 0.0])
@pytest.mark.parametrize("rise", [0.0, 20.0, 41.5, 60.0, 85.0, -50.0])
def test_decode_of_rows_of_one_value(hq, hkv, value, rise):
    """V rows of one value (s = 0) of any size, whose scores rise by `rise` at
    every quarter of the context: weights that meet no scale still must not leave
    fp32's range."""
    n = 400 if hkv == 1 else 3100
    logits = np.repeat([0.0, rise, 2 * rise, 3 * rise], -(-n // 4))[:n]
    got, want, a, spread = _planned(n, hq, hkv, logits, (0, 0.0, value))
    assert (np.abs(got - want) <= _planned_bound(n, a, spread)).all(), (got[0, 0], want[0])
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv", [(2, 1), (8, 1), (128, 32), (256, 32)])
@pytest.mark.parametrize("first", [True, False])
def test_decode_of_rows_of_one_value_among_others(hq, hkv, first):
    """Rows with s = 0 at 2^59 whose weight is 2^-40, and a row of zeros that has
    nearly all of it, at the other end of the context."""
    n = 400 if hkv == 1 else 3100
    at = 0 if first else n - 1
    logits, value = np.zeros(n), np.full(n, 2.0 ** 59)
    logits[at], value[at] = 27.75, 0.0
    got, want, a, spread = _planned(n, hq, hkv, logits, (0, 0.0, value))
    assert (np.abs(got - want) <= _planned_bound(n, a, spread)).all(), (got[0, 0], want[0])
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv", [(2, 1), (8, 1), (128, 32), (256, 32)])
@pytest.mark.parametrize("ratio", [2.0 ** -10, 2.0 ** -16, 2.0 ** -20, 2.0 ** -30])
@pytest.mark.parametrize("at", [0, 37, 399])
def test_decode_of_a_heavy_token_with_small_values(hq, hkv, ratio, at):
    """One token has nearly all the weight and V values far below the others':
    its weight is kept in 22 bits all the same."""
    n = 400 if hkv == 1 else 3100
    logits, s = np.zeros(n), np.full(n, 1.0)
    logits[at], s[at] = 0.6931 * (8 - np.log2(ratio)) + 20, ratio
    got, want, a, spread = _planned(n, hq, hkv, logits, (np.arange(64) % 16, s, -8 * s))
    assert (np.abs(got - want) <= _planned_bound(n, a, spread)).all(), (np.abs(got - want) / a).max()
    assert_clean_status()


@pytest.mark.parametrize("ctx,hq,hkv", [([777], 8, 2), ([3000] * 3, 32, 8), ([2000], 16, 2), ([900] * 40, 64, 8)])
def test_decode_error_in_the_output_norm(ctx, hq, hkv):
    """Random rows: the output is the size of the root of the sum of squares of its
    products, well below the sum that the other bounds are relative to.  In its norm:
    weights in two fp16 parts, 2^-22; exp2, 2^-22; the weights' exponents of up to 6
    (log2), rounded once, 2^-22 ln 2; P V's products of a step cut at 2^-24 of the
    largest, 16 of one sign against a root sum of squares of 4 (the largest 2.5), 10 *
    2^-25; fp32 sums across steps, 2^-23; scores s (q c) + z sum q, four roundings of
    terms of about 5, 2^-24 * 5 * 2 / sqrt(3) as a root mean square; q c's products of
    up to 2.5, cut at 2^-24 in four sums of 16, 2^-24 * 2.5 * sqrt(64) / 2.  In all 2.0
    * 10^-6."""
    got, want, _ = _decode(120 + hq, ctx, hq, hkv, 16)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 2.0 ** -22 * (2 + np.log(2.0)) + 10 * 2.0 ** -25 + 2.0 ** -23 + 2.0 ** -24 * (10 / 3 ** 0.5 + 10), rel
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv,window", [(2, 2, 300), (8, 1, 300), (2, 2, 3000), (8, 1, 3000), (160, 160, 300)])
def test_decode_at_the_longest_context(hq, hkv, window):
    """A context of 2^31 - 128 tokens, nearly all of them behind the window: the
    result of the same last rows at the end of a short context."""
    bs, short = 128, 128 * 24
    tables, nb = C.deal(np.random.default_rng(3), [short], bs)
    rng = np.random.default_rng(4)
    cache = C.random_cache(rng, nb, bs, hkv)
    q = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((1, hq, 64)) * 1.5))
    mb = (2 ** 31 - 128) // bs
    far = torch.full((1, mb), -1, dtype=torch.int32, device=DEV)
    far[0, mb - short // bs:] = _cuda(tables[0])
    out = torch.full((1, hq, 64), float("nan"), device=DEV)
    for cut in (0, 5):
        tvl.kv4_attention_decode(out, C.bf16(q, DEV), _cuda(cache), far,
                                 torch.tensor([2 ** 31 - 128 - cut], dtype=torch.int32, device=DEV), 0.125, window=window)
        want, tol = C.decode_ref(q, tables, [short - cut], 0.125, window, 0, cache=cache)
        assert (np.abs(C.f64(out) - want) <= tol).all(), (np.abs(C.f64(out) - want) / tol).max()
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8), (16, 16)])
@pytest.mark.parametrize("n,top,window", [(200, 900, 0), (200, 900, 300), (600, 120, 0)])
def test_decode_of_more_sequences_than_ctas(hq, hkv, n, top, window):
    """More sequences than CTAs (and than threads of one), whose lengths make most
    CTAs end inside a sequence: one split sequence a CTA in the list to merge."""
    ctx = [int(x) for x in np.random.default_rng(n).integers(0, top, n)]
    got, want, tol = _decode(110 + n, ctx, hq, hkv, 16, window, 3 if window else 0)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert_clean_status()


def test_write_of_rows_of_unlike_magnitude():
    """Where max - z or x - z has more than 24 bits the definition takes it rounded to
    fp32: codes and s are exact from there on, and a value is kept within s / 2 and
    2^-24 of the row's range, 15 s (1 + 2^-7) at most, so 2^-19.9 s."""
    rng = np.random.default_rng(12)
    t, hkv, bs, nb = 64, 4, 16, 6
    x = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((t, hkv, 64)) * 2.0 ** rng.integers(-40, 5, (t, hkv, 64))))
    x[0, 0], x[0, 0, 1], x[0, 0, 2] = 7.5, 15.0, -2.0 ** -30       # range 15 + 2^-30: s = 1
    x[0, 1], x[0, 1, 1], x[0, 1, 2] = 2.0 ** -30, 8.0, -7.0        # x - z = 7 + 2^-30: as 7
    x[0, 2], x[0, 2, 1], x[0, 2, 2] = -0.5, 7.0, 2.0 ** -40
    x[0, 3], x[0, 3, 5] = 2.0 ** -126, -2.0 ** -20
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    cache = torch.zeros(tvl.kv4_cache_shape(nb, hkv, bs), dtype=torch.uint8, device=DEV)
    v = x[::-1].copy()
    tvl.kv4_write(C.bf16(x, DEV), C.bf16(v, DEV), cache, _cuda(slots))
    codes, s, z = C.unpack(cache.cpu().numpy())
    page, off = slots // bs, slots % bs
    for part, rows in ((0, x), (1, v)):
        z0 = rows.min(-1)
        f = lambda y: y.astype(np.float32).astype(np.float64)
        m, e = np.frexp(f(rows.max(-1) - z0) / 15.0)
        s0 = np.ldexp(np.ceil(m * 256.0), e - 8)
        c0 = np.clip(np.where(s0[..., None] > 0, np.rint(f(rows - z0[..., None]) / s0[..., None]), 0), 0, 15)
        assert np.array_equal(z[part][page, off], z0) and np.array_equal(s[part][page, off], s0)
        assert np.array_equal(codes[part][page, off], c0)
        got = s0[..., None] * c0 + z0[..., None]
        assert (np.abs(got - rows) <= s0[..., None] * (0.5 + 2.0 ** -19.9)).all()
    assert s[0][page[0], off[0], 0] == 1.0 and codes[0][page[0], off[0], 0, 0] == 8
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv,n", [(4, 1, 300), (8, 1, 300), (6, 2, 2500), (128, 32, 2500), (224, 32, 2500)])
def test_decode_of_heads_of_unlike_magnitude(hq, hkv, n):
    """Query heads of one group 2^40 apart: each is scaled for itself, so that a small
    one keeps its scores beside a large one (whose softmax has one token)."""
    rng = np.random.default_rng(n + hq)
    tables, nb = C.deal(rng, [n], 16)
    cache = C.random_cache(rng, nb, 16, hkv)
    q = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((1, hq, 64)) * 1.5))
    big = np.arange(hq) % (hq // hkv) == 1
    q[:, big] *= 2.0 ** 40
    out = torch.full((1, hq, 64), float("nan"), device=DEV)
    tvl.kv4_attention_decode(out, C.bf16(q, DEV), _cuda(cache), _cuda(tables), _cuda(np.array([n], np.int32)), 0.125)
    want, tol = C.decode_ref(q, tables, [n], 0.125, 0, 0, cache=cache)
    got = C.f64(out)
    assert (np.abs(got - want) <= tol)[:, ~big].all(), (np.abs(got - want) / tol)[:, ~big].max()
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv,n", [(2, 1, 300), (8, 1, 300), (128, 32, 2500), (256, 32, 2500)])
@pytest.mark.parametrize("size", [2.0 ** 26, 2.0 ** 40, 2.0 ** 90])
def test_decode_of_huge_scores(hq, hkv, n, size):
    """Scores past 2^24, whose differences are whole numbers: the largest one's V row,
    to the parts' 2^-22 and a few fp32 roundings, 2^-20 of 8 s + |z + 8 s|."""
    rng = np.random.default_rng(n + hq)
    tables, nb = C.deal(rng, [n], 16)
    cache = C.random_cache(rng, nb, 16, hkv)
    q = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((1, hq, 64)) * size))
    out = torch.full((1, hq, 64), float("nan"), device=DEV)
    tvl.kv4_attention_decode(out, C.bf16(q, DEV), _cuda(cache), _cuda(tables), _cuda(np.array([n], np.int32)), 0.125)
    codes, ss, zz = C.unpack(cache)
    at = tables[0][np.arange(n) // 16], np.arange(n) % 16
    got = C.f64(out)[0]
    for h in range(hq):
        g = h // (hq // hkv)
        s, z = (x[:, at[0], at[1], g] for x in (ss, zz))
        score = (codes[0][at[0], at[1], g] * s[0][:, None] + z[0][:, None]) @ q[0, h] * 0.125
        j, second = np.argsort(score)[:-3:-1]
        assert score[j] - score[second] > 1e-5 * np.abs(score).max() + 200      # one token, told apart in fp32
        v = codes[1][at[0], at[1], g][j] * s[1][j] + z[1][j]
        assert (np.abs(got[h] - v) <= 2.0 ** -20 * (8 * s[1][j] + abs(z[1][j] + 8 * s[1][j]))).all(), h
    assert_clean_status()
