"""Differential decode attention against the plain form in 64 bits
(tests/diff_common.py derives the bounds)."""
import numpy as np
import pytest
import torch

import diff_common as F
import paged_kv_cache_198_gb300 as tvl
import window_common as C
from gpu_common import DEV, assert_clean_status

pytestmark = pytest.mark.gpu


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _bf(rng, shape, spread=1.0):
    return C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal(shape) * spread))


def _inputs(seed, ctx, hq, hkv, bs, spread=1.0, per_token=False, norm=True):
    rng = np.random.default_rng(seed)
    tables, nb = C.deal(rng, ctx, bs)
    k, v = _bf(rng, (nb, bs, hkv, 64), spread), _bf(rng, (nb, bs, hkv, 64), spread)
    q = _bf(rng, (len(ctx), hq, 64), 1.5)
    lam = rng.uniform(-0.2, 0.9, (len(ctx), hq // 2) if per_token else hq // 2).astype(np.float32)
    weight = _bf(rng, 128) if norm else None
    return tables, k, v, q, lam, weight


def _gpu(q, k, v, tables, ctx, lam, scale, window, sinks, weight, eps, out_scale, **more):
    out = torch.full((q.shape[0], q.shape[1] // 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    tvl.diff_attention_decode(out, C.bf16(q, DEV), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
                              _cuda(np.asarray(ctx, np.int32)), _cuda(lam), scale, window=window, sinks=sinks,
                              norm_weight=None if weight is None else C.bf16(weight, DEV), norm_eps=eps,
                              out_scale=out_scale, **more)
    return out


def _run(seed, ctx, hq, hkv, bs, window=0, sinks=0, spread=1.0, poison=False, scale=0.125, per_token=False,
         norm=True, eps=1e-5, out_scale=0.4):
    tables, k, v, q, lam, weight = _inputs(seed, ctx, hq, hkv, bs, spread, per_token, norm)
    want, tol = F.reference(q, np.arange(len(ctx) + 1), tables, ctx, k, v, lam.astype(np.float64), scale, window,
                            sinks, weight, np.float64(np.float32(eps)), np.float64(np.float32(out_scale)))
    if poison:                      # every slot that is not visible, and the unread table entries
        seen = np.zeros(k.shape[:2], bool)
        for s, n in enumerate(ctx):
            p = C.visible(n - 1, window, sinks) if n else np.zeros(0, int)
            seen[tables[s][p // bs], p % bs] = True
            keep = np.zeros(tables.shape[1], bool)
            keep[p // bs] = True
            tables[s][~keep] = -12345
        k[~seen], v[~seen] = np.nan, np.inf
    got = C.f64(_gpu(q, k, v, tables, ctx, lam, scale, window, sinks, weight, eps, out_scale))
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv,bs", [
    (2, 2, 16), (8, 2, 16), (32, 8, 16), (8, 8, 32), (64, 8, 32), (10, 10, 64), (12, 2, 128), (42, 6, 16),
    (24, 12, 32), (14, 14, 16), (16, 16, 64), (16, 2, 16), (40, 8, 16), (20, 4, 16), (28, 4, 32), (6, 2, 16)])
def test_heads(hq, hkv, bs):
    _run(20 + hq, [1, 700, 16, 17, 333], hq, hkv, bs)


@pytest.mark.parametrize("ctx", [[1], [2], [15], [16], [31, 33], [0, 5, 0], [0], [2000], [64] * 40,
                                 list(range(1, 200, 3)), [7] * 700, [0] * 5, [300] * 3 + [0] * 200])
def test_lengths(ctx):
    _run(40, ctx, 8, 2, 16)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 7), (1, 0), (1, 1), (16, 0), (17, 4), (100, 16),
                                          (100, 17), (64, 1000), (5000, 4), (640, 300)])
@pytest.mark.parametrize("bs", [16, 64])
def test_windows_with_poisoned_unseen_slots(window, sinks, bs):
    _run(50, [1, 90, 0, 101, 1500, 640, 116], 12, 6, bs, window, sinks, poison=True)


@pytest.mark.parametrize("spread", [1e-6, 1e4])
@pytest.mark.parametrize("norm", [False, True])
def test_magnitudes(spread, norm):
    _run(60, [500, 77], 16, 4, 16, spread=spread, norm=norm, scale=0.125 / max(1.0, spread))


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_scales(scale):
    _run(61, [300, 40, 1], 8, 4, 16, scale=scale)


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("norm,eps,out_scale", [(True, 1e-5, 0.4), (True, 0.0, 1.0), (True, 1.0, -2.0),
                                                (False, 0.0, 1.0), (False, 1e-5, 0.25)])
def test_lambda_and_norm(per_token, norm, eps, out_scale):
    _run(62, [200, 0, 33, 900], 16, 4, 32, per_token=per_token, norm=norm, eps=eps, out_scale=out_scale)


def test_a_difference_of_zero_is_a_zero_row():
    """Equal maps and lambda 1: d is 0 up to nothing at all (the two maps take the
    same operations on the same values), with and without eps."""
    tables, k, v, q, _, weight = _inputs(63, [300, 1], 8, 4, 16)
    k[:, :, 1::2] = k[:, :, 0::2]
    q[:, 1::2] = q[:, 0::2]
    for eps in (0.0, 1e-5):
        out = _gpu(q, k, v, tables, [300, 1], np.ones(4, np.float32), 0.125, 0, 0, weight, eps, 1.0)
        assert (C.f64(out) == 0).all()
    assert_clean_status()


def test_lambda_zero_is_plain_attention_over_both_halves():
    """Against paged_attention_decode of the even heads, whose keys are the even KV
    heads and whose values are either V head: within both bounds."""
    ctx = [900, 3, 0, 1777]
    tables, k, v, q, _, _ = _inputs(64, ctx, 16, 4, 16)
    got = C.f64(_gpu(q, k, v, tables, ctx, np.zeros(8, np.float32), 0.125, 0, 0, None, 0.0, 1.0))
    want, tol = F.reference(q, np.arange(5), tables, ctx, k, v, np.zeros(8), 0.125)
    for half in (0, 1):
        o = torch.empty(4, 8, 64, device=DEV)
        kk, vv = k[:, :, 0::2], v[:, :, half::2]
        tvl.paged_attention_decode(o, C.bf16(q[:, 0::2], DEV), C.bf16(kk, DEV), C.bf16(vv, DEV), _cuda(tables),
                                   _cuda(np.asarray(ctx, np.int32)), 0.125)
        mine = got[:, :, 64 * half:64 * half + 64]
        assert (np.abs(C.f64(o) - mine) <= 2 * tol[:, :, 64 * half:64 * half + 64]).all()
    assert_clean_status()


def test_repeats_bit_for_bit_and_from_two_graphs_of_one_workspace():
    ctx = [3, 900, 0, 450, 77]
    tables, k, v, q, lam, weight = _inputs(65, ctx, 32, 8, 16)
    a = [C.bf16(x, DEV) for x in (q, k, v)] + [_cuda(tables), _cuda(np.asarray(ctx, np.int32)), _cuda(lam), 0.125]
    ws = torch.empty(tvl.diff_decode_workspace_size(32, 8), dtype=torch.uint8, device=DEV)
    w = C.bf16(weight, DEV)
    outs = [torch.full((5, 16, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    for i, win in ((0, 0), (1, 500)):
        tvl.diff_attention_decode(outs[i], *a, window=win, sinks=2, norm_weight=w)
    graphs = []
    for i, win in ((2, 0), (3, 500)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tvl.diff_attention_decode(outs[i], *a, window=win, sinks=2, norm_weight=w, workspace=ws)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert_clean_status()


@pytest.mark.parametrize("seed", range(16))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(900 + seed)
    kvp, g = int(rng.integers(1, 9)), int(rng.integers(1, 9))
    n = int(rng.integers(1, 9))
    ctx = [int(x) for x in np.exp(rng.uniform(0, np.log(1500), n))]
    _run(1000 + seed, ctx, 2 * kvp * g, 2 * kvp, int(rng.choice([16, 32, 64, 128])),
         int(rng.integers(1, 800)) if seed & 2 else 0, int(rng.integers(0, 70)), poison=bool(seed & 1),
         per_token=bool(seed & 4), norm=seed % 3 != 0)


def test_rising_scores_move_the_reference():
    """Scores that rise by some 40 along the context, on the two maps in opposite
    directions."""
    ctx = [1200]
    tables, k, v, q, lam, weight = _inputs(66, ctx, 8, 2, 16)
    q[:] = 1.0
    ramp = np.linspace(-2.5, 2.5, 1200)
    pos = np.arange(1200)
    k[tables[0][pos // 16], pos % 16, 0] = ramp[:, None]
    k[tables[0][pos // 16], pos % 16, 1] = -ramp[:, None]
    k = C.bf16_to_f64(C.f64_to_bf16_bits(k))
    want, tol = F.reference(q, [0, 1], tables, ctx, k, v, lam.astype(np.float64), 0.25, weight=weight,
                            eps=np.float64(np.float32(1e-5)))
    got = C.f64(_gpu(q, k, v, tables, ctx, lam, 0.25, 0, 0, weight, 1e-5, 1.0))
    assert (np.abs(got - want) <= tol).all()
    assert_clean_status()


def test_bad_block_ids_and_lengths_are_reported():
    ctx = [40, 20]
    tables, k, v, q, lam, weight = _inputs(67, ctx, 8, 2, 16)
    good = _gpu(q, k, v, tables, ctx, lam, 0.125, 0, 0, weight, 1e-5, 1.0)
    bad = tables.copy()
    bad[0, 1] = k.shape[0]
    out = _gpu(q, k, v, bad, ctx, lam, 0.125, 0, 0, weight, 1e-5, 1.0)
    assert tvl.get_device_status() == tvl.DEV_BAD_BLOCK_ID and torch.equal(out[1], good[1])
    _gpu(q, k, v, tables[:, :2].copy(), [-3, 20], lam, 0.125, 0, 0, weight, 1e-5, 1.0)
    assert tvl.get_device_status() == tvl.DEV_BAD_CONTEXT_LEN
