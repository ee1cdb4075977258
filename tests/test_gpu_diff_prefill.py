"""Differential prefill attention against the plain form in 64 bits
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


def _inputs(seed, prefix, new, hq, hkv, bs, spread=1.0, per_token=False, norm=True):
    rng = np.random.default_rng(seed)
    ctx = [p + n for p, n in zip(prefix, new)]
    tables, nb = C.deal(rng, ctx, bs)
    k, v = _bf(rng, (nb, bs, hkv, 64), spread), _bf(rng, (nb, bs, hkv, 64), spread)
    t = sum(new)
    q = _bf(rng, (t, hq, 64), 1.5)
    lam = rng.uniform(-0.2, 0.9, (t, hq // 2) if per_token else hq // 2).astype(np.float32)
    weight = _bf(rng, 128) if norm else None
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return ctx, tables, k, v, q, lam, weight, starts


def _gpu(q, starts, k, v, tables, ctx, lam, scale, max_q, window, sinks, weight, eps, out_scale, **more):
    out = torch.full((q.shape[0], q.shape[1] // 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    tvl.diff_attention_prefill(out, C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
                               _cuda(np.asarray(ctx, np.int32)), _cuda(lam), scale, max_q, window=window,
                               sinks=sinks, norm_weight=None if weight is None else C.bf16(weight, DEV),
                               norm_eps=eps, out_scale=out_scale, **more)
    return out


def _run(seed, prefix, new, hq, hkv, bs, window=0, sinks=0, spread=1.0, poison=False, scale=0.125,
         per_token=False, norm=True, eps=1e-5, out_scale=0.4):
    ctx, tables, k, v, q, lam, weight, starts = _inputs(seed, prefix, new, hq, hkv, bs, spread, per_token, norm)
    want, tol = F.reference(q, starts, tables, ctx, k, v, lam.astype(np.float64), scale, window, sinks, weight,
                            np.float64(np.float32(eps)), np.float64(np.float32(out_scale)), bits=11, prefill=True)
    if poison:                      # every slot that no row sees, and the unread table entries
        seen = np.zeros(k.shape[:2], bool)
        for s, n in enumerate(ctx):
            for p0 in range(n - new[s], n):
                p = C.visible(p0, window, sinks)
                seen[tables[s][p // bs], p % bs] = True
            tables[s][-(-n // bs):] = -12345
        k[~seen], v[~seen] = np.nan, np.inf
    got = C.f64(_gpu(q, starts, k, v, tables, ctx, lam, scale, max(new), window, sinks, weight, eps, out_scale))
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert_clean_status()


@pytest.mark.parametrize("new", [[1], [2], [15], [16], [17], [63, 64, 65], [127], [128], [129], [200, 1, 0, 31]])
@pytest.mark.parametrize("prefix", [0, 37])
def test_chunk_lengths(new, prefix):
    _run(1, [prefix] * len(new), new, 4, 2, 16)


@pytest.mark.parametrize("hq,hkv,bs", [(2, 2, 16), (8, 2, 32), (16, 4, 64), (16, 2, 128), (12, 4, 16), (6, 2, 32),
                                       (10, 2, 16), (14, 14, 64), (8, 8, 128)])
def test_heads_and_block_sizes(hq, hkv, bs):
    _run(2, [100, 0, 250], [40, 20, 33], hq, hkv, bs)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 9), (1, 0), (1, 1), (16, 4), (64, 0), (100, 17), (300, 70),
                                          (5000, 4), (40, 1000)])
@pytest.mark.parametrize("bs", [16, 128])
def test_windows_with_poisoned_unseen_slots(window, sinks, bs):
    _run(3, [500, 0, 77], [60, 150, 3], 4, 2, bs, window, sinks, poison=True)


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("norm,eps,out_scale", [(True, 1e-5, 0.4), (True, 0.0, 1.0), (True, 1.0, -2.0),
                                                (False, 0.0, 1.0), (False, 1e-5, 0.25)])
def test_lambda_and_norm(per_token, norm, eps, out_scale):
    _run(4, [60, 0], [70, 35], 8, 2, 16, per_token=per_token, norm=norm, eps=eps, out_scale=out_scale)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_scales(scale):
    _run(5, [90], [50], 4, 2, 16, scale=scale)


@pytest.mark.parametrize("spread", [1e-3, 1e3])
def test_magnitudes(spread):
    _run(6, [120], [40], 4, 2, 16, spread=spread, scale=0.125 / max(1.0, spread))


def test_more_units_than_ctas_and_than_ranks():
    """Several units a CTA, empty and short sequences, and more query tiles than are
    ranked (600 items)."""
    _run(7, [30] * 40, [5, 0, 130, 1, 64] * 8, 8, 2, 16)
    _run(8, [3] * 600, [1] * 300 + [2] * 300, 4, 2, 16)


def test_rising_and_falling_scores_move_the_reference():
    """Scores that rise by some 30 along the context on one map and fall on the other."""
    ctx, tables, k, v, q, lam, weight, starts = _inputs(9, [700], [90], 4, 2, 16)
    q[:] = 1.0
    pos = np.arange(790)
    ramp = np.linspace(-2.0, 2.0, 790)
    k[tables[0][pos // 16], pos % 16, 0] = ramp[:, None]
    k[tables[0][pos // 16], pos % 16, 1] = -ramp[:, None]
    k = C.bf16_to_f64(C.f64_to_bf16_bits(k))
    want, tol = F.reference(q, starts, tables, ctx, k, v, lam.astype(np.float64), 0.125, weight=weight,
                            eps=np.float64(np.float32(1e-5)), bits=11, prefill=True)
    got = C.f64(_gpu(q, starts, k, v, tables, ctx, lam, 0.125, 90, 0, 0, weight, 1e-5, 1.0))
    assert (np.abs(got - want) <= tol).all()
    assert_clean_status()


def test_a_difference_of_zero_is_a_zero_row():
    ctx, tables, k, v, q, _, weight, starts = _inputs(10, [40, 0], [150, 7], 8, 4, 16)
    k[:, :, 1::2] = k[:, :, 0::2]
    q[:, 1::2] = q[:, 0::2]
    for eps in (0.0, 1e-5):
        out = _gpu(q, starts, k, v, tables, ctx, np.ones(4, np.float32), 0.125, 150, 0, 0, weight, eps, 1.0)
        assert (C.f64(out) == 0).all()
    assert_clean_status()


def test_the_last_row_agrees_with_the_decode():
    ctx, tables, k, v, q, lam, weight, starts = _inputs(11, [300, 20, 0], [40, 1, 5], 16, 4, 32)
    a = dict(window=100, sinks=4)
    got = C.f64(_gpu(q, starts, k, v, tables, ctx, lam, 0.125, 40, *a.values(), weight, 1e-5, 0.5))
    last = starts[1:] - 1
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    tvl.diff_attention_decode(out, C.bf16(q[last], DEV), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
                              _cuda(np.asarray(ctx, np.int32)), _cuda(lam), 0.125, **a,
                              norm_weight=C.bf16(weight, DEV), out_scale=0.5)
    _, tol = F.reference(q, starts, tables, ctx, k, v, lam.astype(np.float64), 0.125, 100, 4, weight,
                         np.float64(np.float32(1e-5)), 0.5, bits=11, prefill=True)
    assert (np.abs(got[last] - C.f64(out)) <= 2 * tol[last]).all()
    assert_clean_status()


def test_repeats_bit_for_bit_captured_and_on_another_stream():
    ctx, tables, k, v, q, lam, weight, starts = _inputs(12, [100, 0, 40], [140, 33, 1], 16, 4, 16)
    args = [C.bf16(q, DEV), _cuda(starts), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
            _cuda(np.asarray(ctx, np.int32)), _cuda(lam), 0.125, 140]
    w = C.bf16(weight, DEV)
    outs = [torch.full((174, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    tvl.diff_attention_prefill(outs[0], *args, norm_weight=w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    tvl.diff_attention_prefill(outs[1], *args, norm_weight=w, stream=side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tvl.diff_attention_prefill(outs[2], *args, norm_weight=w)
    outs[2].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert_clean_status()


def test_inconsistent_lengths_are_reported_and_their_rows_left():
    ctx, tables, k, v, q, lam, weight, starts = _inputs(13, [20, 30, 10], [5, 40, 7], 4, 2, 16)
    good = _gpu(q, starts, k, v, tables, ctx, lam, 0.125, 40, 0, 0, weight, 1e-5, 1.0)
    for bad_ctx, bit in ((39, tvl.DEV_BAD_QUERY_LEN), (tables.shape[1] * 16 + 1, tvl.DEV_BAD_CONTEXT_LEN)):
        out = _gpu(q, starts, k, v, tables, [ctx[0], bad_ctx, ctx[2]], lam, 0.125, 40, 0, 0, weight, 1e-5, 1.0)
        assert tvl.get_device_status() == bit
        assert torch.equal(out[:5], good[:5]) and torch.equal(out[45:], good[45:]) and out[5:45].isnan().all()
    bad = tables.copy()
    bad[1, 2] = k.shape[0] + 7
    out = _gpu(q, starts, k, v, bad, ctx, lam, 0.125, 40, 0, 0, weight, 1e-5, 1.0)
    assert tvl.get_device_status() == tvl.DEV_BAD_BLOCK_ID
    assert torch.equal(out[:5], good[:5]) and torch.equal(out[45:], good[45:])


def test_a_value_past_fp16_is_reported_where_it_is_seen():
    ctx, tables, k, v, q, lam, weight, starts = _inputs(14, [300], [10], 2, 2, 16)
    v[tables[0][50 // 16], 50 % 16] = 1e6
    _gpu(q, starts, k, v, tables, ctx, lam, 0.125, 10, 0, 0, weight, 1e-5, 1.0)
    assert tvl.get_device_status() == tvl.DEV_NONFINITE
    assert np.isfinite(C.f64(_gpu(q, starts, k, v, tables, ctx, lam, 0.125, 10, 64, 4, weight, 1e-5, 1.0))).all()
    assert_clean_status()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(500 + seed)
    n = int(rng.integers(1, 6))
    kvp, g = int(rng.integers(1, 4)), int(rng.integers(1, 9))
    while kvp * g > 8:
        g = max(1, g // 2)
    new = [int(x) for x in np.exp(rng.uniform(0, np.log(250), n))]
    prefix = [int(x) for x in rng.integers(0, 400, n)]
    _run(600 + seed, prefix, new, 2 * kvp * g, 2 * kvp, int(rng.choice([16, 32, 64, 128])),
         int(rng.integers(1, 300)) if seed & 2 else 0, int(rng.integers(0, 70)), poison=bool(seed & 1),
         per_token=bool(seed & 4), norm=seed % 3 != 0)
