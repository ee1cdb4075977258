"""Chunked prefill with a sliding window and sinks, against the plain form in
64 bits.

Bound, per output element, with A, B, n as in tests/window_common.py and M =
max |v|: P is rounded to fp16 (2^-11 relative, 2^-25 absolute below 2^-14, and
the row's sum is at least 1 in the same units), V to fp16 (exact, or 2^-25
absolute), scores and sums as in the decode:
  A (2^-11 + 2 (80 * 2^-24 B + 2^-21) + (n / 16 + 64) 2^-23) + n 2^-25 M + 2^-25,
then the output is rounded to bf16: 2^-8 of its value more."""
import numpy as np
import pytest
import torch

import paged_kv_cache_198_gb300 as tvl
import window_common as C
from gpu_common import DEV, assert_clean_status

pytestmark = pytest.mark.gpu


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _bf(rng, shape, spread=1.0):
    return C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal(shape) * spread))


def _ref(q, k, v, tables, ctx, new, scale, window, sinks):
    bs, hkv = k.shape[1], k.shape[2]
    g = q.shape[1] // hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    at = 0
    for s, (n, m) in enumerate(zip(ctx, new)):
        pos = np.arange(n)
        kk, vv = (x[tables[s][pos // bs], pos % bs] for x in (k, v))
        p = np.arange(n - m, n)[:, None]
        ok = pos <= p
        if window:
            ok &= (pos > p - window) | (pos < sinks)
        cnt = ok.sum(1)[:, None]
        for h in range(q.shape[1]):
            x = q[at:at + m, h] @ kk[:, h // g].T * scale
            b = np.where(ok, np.abs(q[at:at + m, h]) @ np.abs(kk[:, h // g]).T * abs(scale), 0).max(1)[:, None]
            x = np.where(ok, x, -np.inf)
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            o = w @ vv[:, h // g]
            a = w @ np.abs(vv[:, h // g])
            big = np.abs(vv[:, h // g]).max()
            t = (a * (2.0 ** -11 + 2 * (80 * 2.0 ** -24 * b + 2.0 ** -21) + (cnt / 16 + 64) * 2.0 ** -23)
                 + cnt * 2.0 ** -25 * big + 2.0 ** -25)
            out[at:at + m, h] = o
            tol[at:at + m, h] = t * (1 + 2.0 ** -8) + np.abs(o) * 2.0 ** -8
        at += m
    return out, tol


def _setup(seed, ctx, new, hq, hkv, bs, spread=1.0):
    rng = np.random.default_rng(seed)
    tables, nb = C.deal(rng, ctx, bs)
    k, v = _bf(rng, (nb, bs, hkv, 64), spread), _bf(rng, (nb, bs, hkv, 64), spread)
    q = _bf(rng, (sum(new), hq, 64), 1.5)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return rng, tables, nb, k, v, q, starts


def _run(seed, ctx, new, hq, hkv, bs, window, sinks, spread=1.0, poison=False, extra_rows=0, scale=0.125):
    rng, tables, nb, k, v, q, starts = _setup(seed, ctx, new, hq, hkv, bs, spread)
    want, tol = _ref(q, k, v, tables, ctx, new, scale, window, sinks)
    if poison:
        seen = np.zeros((nb, bs), bool)
        for s, (n, m) in enumerate(zip(ctx, new)):
            need = np.zeros(tables.shape[1], bool)
            for p in {n - m, n - 1} if m else ():
                j = C.visible(p, window, sinks)
                seen[tables[s][j // bs], j % bs] = True
                need[j // bs] = True
            lo, hi = (n - m - window + 1, n) if window else (0, n)
            j = np.arange(max(0, lo), hi) if m else np.arange(0)
            seen[tables[s][j // bs], j % bs] = True
            need[j // bs] = True
            tables[s][~need] = -7
        k[~seen], v[~seen] = np.nan, np.nan
    out = torch.full((q.shape[0] + extra_rows, hq, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    qq = np.concatenate([q, np.zeros((extra_rows, hq, 64))]) if extra_rows else q
    tvl.paged_attention_window_prefill(out, C.bf16(qq, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV),
                                       _cuda(tables), _cuda(np.asarray(ctx, np.int32)), scale, max(new + [1]),
                                       window, sinks=sinks)
    got = C.f64(out)
    t = q.shape[0]
    assert np.isfinite(got).all()
    assert (np.abs(got[:t] - want) <= tol).all(), (np.abs(got[:t] - want) / np.maximum(tol, 1e-30)).max()
    assert (got[t:] == 9.0).all()
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv,bs", [(8, 2, 16), (32, 8, 16), (4, 4, 32), (16, 8, 64), (8, 1, 128), (2, 1, 16)])
def test_heads(hq, hkv, bs):
    _run(10 + hq, [300, 17, 500], [200, 17, 1], hq, hkv, bs, 100, 4)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 9), (1, 0), (1, 1), (16, 0), (64, 4), (100, 17), (127, 0),
                                          (128, 128), (129, 300), (1000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("bs", [16, 128])
def test_windows_with_poisoned_unseen_slots(window, sinks, bs):
    _run(30, [700, 129, 1, 260], [150, 129, 1, 130], 4, 2, bs, window, sinks, poison=True)


@pytest.mark.parametrize("ctx,new", [([1], [1]), ([128], [128]), ([129], [129]), ([5, 5, 5], [5, 0, 5]),
                                     ([900], [1]), ([400] * 20, [3] * 20), ([1000, 640], [513, 640])])
def test_lengths(ctx, new):
    _run(50, ctx, new, 8, 2, 16, 70, 3)


def test_a_window_that_leaves_a_first_tile_empty_for_late_rows():
    """Without sinks the first key tile holds no key of the late rows, whose
    scores later are far below zero: the reference is set where keys appear."""
    rng, tables, nb, k, v, q, starts = _setup(60, [600], [300], 4, 2, 16)
    k[..., 0] = -40.0
    q[..., 0] = 30.0                       # every score near -150
    want, tol = _ref(q, k, v, tables, [600], [300], 0.125, 20, 0)
    out = torch.empty(300, 4, 64, dtype=torch.bfloat16, device=DEV)
    tvl.paged_attention_window_prefill(out, C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV),
                                       _cuda(tables), _cuda(np.array([600], np.int32)), 0.125, 300, 20)
    assert (np.abs(C.f64(out) - want) <= tol).all()
    assert_clean_status()


def test_rows_behind_the_last_sequence_stay():
    _run(61, [40, 200], [40, 60], 8, 2, 16, 30, 2, extra_rows=13)


def test_without_a_window_it_is_the_plain_prefill_rounded_to_bf16():
    rng, tables, nb, k, v, q, starts = _setup(62, [900, 300, 77], [400, 300, 1], 32, 8, 16)
    args = [C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
            _cuda(np.array([900, 300, 77], np.int32)), 0.125, 400]
    a = torch.empty(701, 32, 64, device=DEV)
    b = torch.empty(701, 32, 64, dtype=torch.bfloat16, device=DEV)
    tvl.paged_attention_prefill(a, *args)
    tvl.paged_attention_window_prefill(b, *args, 0)
    assert torch.equal(a.to(torch.bfloat16), b)


def test_one_row_prefill_agrees_with_the_windowed_decode():
    ctx = [33, 700, 5]
    rng, tables, nb, k, v, q, starts = _setup(63, ctx, [1, 1, 1], 8, 2, 16)
    kv = [C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables), _cuda(np.array(ctx, np.int32)), 0.125]
    a = torch.empty(3, 8, 64, device=DEV)
    b = torch.empty(3, 8, 64, dtype=torch.bfloat16, device=DEV)
    tvl.paged_attention_window_decode(a, C.bf16(q, DEV), *kv, 50, sinks=4)
    tvl.paged_attention_window_prefill(b, C.bf16(q, DEV), _cuda(starts), *kv, 1, 50, sinks=4)
    _, tol = _ref(q, k, v, tables, ctx, [1, 1, 1], 0.125, 50, 4)
    assert (np.abs(C.f64(a) - C.f64(b)) <= 2 * tol).all()


def test_nonfinite_v_is_reported_and_stays_in_its_tiles():
    """A NaN V row at position 3 (no sink): rows of later tiles, whose windows
    have left it behind, are as without it."""
    rng, tables, nb, k, v, q, starts = _setup(64, [600], [600], 4, 2, 16)
    want, tol = _ref(q, k, v, tables, [600], [600], 0.125, 32, 0)
    v[tables[0][0], 3] = np.nan
    out = torch.empty(600, 4, 64, dtype=torch.bfloat16, device=DEV)
    tvl.paged_attention_window_prefill(out, C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV),
                                       _cuda(tables), _cuda(np.array([600], np.int32)), 0.125, 600, 32)
    assert tvl.get_device_status() == tvl.DEV_NONFINITE
    got = C.f64(out)
    assert (np.abs(got - want) <= tol)[256:].all()
    assert np.isnan(got[3]).all()


def test_bad_lengths_are_reported_and_left_unwritten():
    rng, tables, nb, k, v, q, starts = _setup(65, [60, 60], [20, 20], 4, 2, 16)
    out = torch.full((40, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    tvl.paged_attention_window_prefill(out, C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV),
                                       _cuda(tables), _cuda(np.array([10, 60], np.int32)), 0.125, 20, 8)
    assert tvl.get_device_status() == tvl.DEV_BAD_QUERY_LEN
    assert (C.f64(out)[:20] == 9.0).all() and (C.f64(out)[20:] != 9.0).any()


def test_captured_and_replayed():
    rng, tables, nb, k, v, q, starts = _setup(66, [300, 90], [100, 90], 8, 2, 16)
    args = [C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
            _cuda(np.array([300, 90], np.int32)), 0.125, 100, 64]
    a, b = (torch.empty(190, 8, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tvl.paged_attention_window_prefill(a, *args, sinks=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tvl.paged_attention_window_prefill(b, *args, sinks=4)
    b.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_prefill_over_a_4bit_prefix():
    """A chunk on a prefix held in 4 bits: write, expand the blocks, prefill
    with a window, all through the allocator's slots and tables."""
    rng = np.random.default_rng(67)
    hq, hkv, bs, nb = 8, 2, 16, 40
    alloc = tvl.BlockAllocator(nb, bs)
    cache = torch.zeros(tvl.kv4_cache_shape(nb, hkv, bs), dtype=torch.uint8, device=DEV)
    kc = torch.zeros(nb, bs, hkv, 64, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    seq = alloc.new_sequence()
    for n in (150, 83):
        slots = alloc.append(seq, n)
        k, v, q = (C.bf16(rng.standard_normal((n, h, 64)), DEV) for h in (hkv, hkv, hq))
        tvl.kv4_write(k, v, cache, _cuda(slots))
        tables, ctx = alloc.build_tables([seq], 20)
        used = _cuda(tables[0][:-(-int(ctx[0]) // bs)])
        tvl.kv4_expand_blocks(kc, vc, cache, used, used)
        out = torch.empty(n, hq, 64, dtype=torch.bfloat16, device=DEV)
        tvl.paged_attention_window_prefill(out, q, _cuda(np.array([0, n], np.int32)), kc, vc, _cuda(tables),
                                           _cuda(ctx), 0.125, n, 100, sinks=4)
        want, tol = _ref(C.f64(q), C.f64(kc), C.f64(vc), tables, [int(ctx[0])], [n], 0.125, 100, 4)
        assert (np.abs(C.f64(out) - want) <= tol).all()
    assert_clean_status()


@pytest.mark.parametrize("seed", range(8))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(700 + seed)
    hkv, g = int(rng.integers(1, 6)), int(rng.choice([1, 2, 4, 8]))
    n = int(rng.integers(1, 6))
    new = [int(x) for x in np.exp(rng.uniform(0, np.log(400), n))]
    ctx = [m + int(rng.integers(0, 500)) for m in new]
    _run(800 + seed, ctx, new, hkv * g, hkv, int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 500)),
         int(rng.integers(0, 200)), poison=bool(seed & 1))


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1e-42, -1e-42, 1.0])
@pytest.mark.parametrize("hkv", [2, 8])
def test_scales(scale, hkv):
    """Masked scores are infinities against the scale's sign; a scale of nothing
    must not turn them into NaN."""
    _run(70, [300, 140], [200, 140], 8, hkv, 16, 100, 4, scale=scale)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 0), (100, 4)])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (32, 8)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e5])
def test_v_of_a_later_token_leaves_the_earlier_tiles(window, sinks, hq, hkv, value):
    """Rows 400 .. 699 in tiles of 128 rows: a V at position 530 that fp16 does not
    hold is seen by no row of the first tile (400 .. 527), whose last key tile
    reaches past it; its rows equal those without it bit for bit."""
    rng, tables, nb, k, v, q, starts = _setup(72, [700], [300], hq, hkv, 16)
    k, q = C.bf16(k, DEV), C.bf16(q, DEV)
    outs = []
    for x in (None, value):
        if x is not None:
            v[tables[0][530 // 16], 530 % 16] = x
        outs.append(torch.empty(300, hq, 64, dtype=torch.bfloat16, device=DEV))
        tvl.paged_attention_window_prefill(outs[-1], q, _cuda(starts), k, C.bf16(v, DEV), _cuda(tables),
                                           _cuda(np.array([700], np.int32)), 0.125, 300, window, sinks=sinks)
    assert tvl.get_device_status() == tvl.DEV_NONFINITE
    assert torch.equal(outs[0][:128], outs[1][:128])
    assert not torch.isfinite(outs[1][130:131]).all()
    if window == 0:              # and so in the plain form
        plain = torch.empty(300, hq, 64, device=DEV)
        tvl.paged_attention_prefill(plain, q, _cuda(starts), k, C.bf16(v, DEV), _cuda(tables),
                                    _cuda(np.array([700], np.int32)), 0.125, 300)
        assert tvl.get_device_status() == tvl.DEV_NONFINITE
        assert torch.equal(plain[:128].to(torch.bfloat16), outs[0][:128])


def test_repeats_bit_for_bit():
    """More units than SMs, of different lengths: the same call again, and again
    among other work."""
    ctx, new = [900, 300, 77, 1500] * 4, [400, 300, 1, 513] * 4
    rng, tables, nb, k, v, q, starts = _setup(73, ctx, new, 32, 8, 16)
    args = [C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
            _cuda(np.array(ctx, np.int32)), 0.125, 513, 200]
    outs = [torch.empty(sum(new), 32, 64, dtype=torch.bfloat16, device=DEV) for _ in range(6)]
    for o in outs:
        tvl.paged_attention_window_prefill(o, *args, sinks=4)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert_clean_status()


def test_pools_past_32_bit_offsets():
    """Blocks at both ends of a 4-bit pool of 5 GB and bf16 pools of 9.5 GB each: write,
    decode, copy, expansion, and decode and prefill over the expanded blocks."""
    rng = np.random.default_rng(74)
    hq, hkv, bs, n = 32, 8, 16, 700
    nb = 5 * 2 ** 30 // (bs * hkv * 72)
    cache = torch.zeros(tvl.kv4_cache_shape(nb, hkv, bs), dtype=torch.uint8, device=DEV)
    kc, vc = (torch.empty(nb, bs, hkv, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ids = np.concatenate([nb - 1 - np.arange(0, 40, 2), [0, 1], nb // 2 + np.arange(22)]).astype(np.int32)
    pos = np.arange(n)
    k, v = (C.bf16(_bf(rng, (n, hkv, 64)), DEV) for _ in range(2))
    q = _bf(rng, (n, hq, 64), 1.5)
    tables, ln = _cuda(ids[None]), _cuda(np.array([n], np.int32))
    tvl.kv4_write(k, v, cache, _cuda((ids[pos // bs].astype(np.int64) * bs + pos % bs).astype(np.int32)))
    small = cache[_cuda(ids).long()].cpu().numpy()
    here = np.arange(len(ids), dtype=np.int32)[None]
    codes, s, z = C.unpack(small)
    c0, s0, z0 = C.quantise(C.f64(v))
    assert np.array_equal(codes[1][pos // bs, pos % bs], c0) and np.array_equal(z[1][pos // bs, pos % bs], z0)

    def check_decode(window, call, **ref):
        out = torch.full((1, hq, 64), float("nan"), device=DEV)
        call(out, C.bf16(q[-1:], DEV))
        want, tol = C.decode_ref(q[-1:], here, [n], 0.125, window, 0, **ref)
        assert (np.abs(C.f64(out) - want) <= tol).all()

    check_decode(0, lambda o, x: tvl.kv4_attention_decode(o, x, cache, tables, ln, 0.125), cache=small)
    tvl.kv4_copy_blocks(cache, _cuda(ids[:2]), _cuda(np.array([nb - 2, 7], np.int32)))
    assert torch.equal(cache[nb - 2], cache[int(ids[0])]) and torch.equal(cache[7], cache[int(ids[1])])
    tvl.kv4_expand_blocks(kc, vc, cache, _cuda(ids), _cuda(ids))
    big = C.f64(kc[_cuda(ids).long()]), C.f64(vc[_cuda(ids).long()])
    val = C.values(small)
    seen = (np.arange(len(ids))[:, None] * bs + np.arange(bs))[..., None, None] < n
    for got, want in zip(big, val):
        assert (np.where(seen, np.abs(got - want), 0) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -20).all()
    big = [np.where(seen, x, 0) for x in big]
    check_decode(100, lambda o, x: tvl.paged_attention_window_decode(o, x, kc, vc, tables, ln, 0.125, 100), kv=big)
    out = torch.empty(300, hq, 64, dtype=torch.bfloat16, device=DEV)
    tvl.paged_attention_window_prefill(out, C.bf16(q[-300:], DEV), _cuda(np.array([0, 300], np.int32)), kc, vc, tables,
                                       ln, 0.125, 300, 200, sinks=4)
    want, tol = _ref(q[-300:], *big, here, [n], [300], 0.125, 200, 4)
    assert (np.abs(C.f64(out) - want) <= tol).all()
    assert_clean_status()
