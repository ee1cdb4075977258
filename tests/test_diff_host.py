"""Differential attention without a GPU: refusals of the C ABI (before any CUDA
call) and of the binding, and the plain form against closed forms."""
import numpy as np
import pytest
import torch

import diff_common as F


@pytest.fixture(scope="module")
def tvl():
    from paged_kv_cache_198_gb300 import _build

    _build.build()
    import paged_kv_cache_198_gb300 as t

    return t


D16 = 256      # a well aligned stand-in for a device pointer; never read


def _decode(t, **k):
    a = dict(out=D16, q=D16, kc=D16, vc=D16, tab=D16, ctx=D16, lam=D16, per=0, w=D16, eps=1e-5, osc=1.0,
             s=4, hq=8, hkv=2, d=64, bs=16, nb=64, mb=8, scale=0.125, window=0, sinks=0, ws=D16, wsb=1 << 30)
    a.update(k)
    return t._load().tvl_diff_attention_decode(*a.values(), None)


@pytest.mark.parametrize("bad,want", [
    (dict(s=-1), "INVALID_ARG"), (dict(d=128), "UNSUPPORTED"), (dict(bs=24), "UNSUPPORTED"),
    (dict(hq=9), "INVALID_ARG"), (dict(hq=9, hkv=3), "INVALID_ARG"), (dict(hq=8, hkv=1), "INVALID_ARG"),
    (dict(hq=18, hkv=2), "UNSUPPORTED"), (dict(hkv=0), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"),
    (dict(mb=0), "INVALID_ARG"), (dict(nb=1 << 27), "UNSUPPORTED"), (dict(mb=1 << 27), "UNSUPPORTED"),
    (dict(window=-1), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(q=D16 + 8), "INVALID_ARG"),
    (dict(kc=None), "INVALID_ARG"), (dict(vc=D16 + 2), "INVALID_ARG"), (dict(tab=None), "INVALID_ARG"),
    (dict(ctx=None), "INVALID_ARG"), (dict(lam=None), "INVALID_ARG"), (dict(lam=D16 + 2), "INVALID_ARG"),
    (dict(w=D16 + 8), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(eps=float("inf")), "INVALID_ARG"), (dict(osc=float("inf")), "INVALID_ARG"),
    (dict(ws=None), "WORKSPACE"), (dict(ws=D16 + 8), "INVALID_ARG")])
def test_decode_refusals(tvl, bad, want):
    assert _decode(tvl, **bad) == getattr(tvl, "ERR_" + want)
    assert tvl._load().tvl_last_error()


def _prefill(t, **k):
    a = dict(out=D16, q=D16, qsl=D16, kc=D16, vc=D16, tab=D16, ctx=D16, lam=D16, per=0, w=D16, eps=1e-5,
             osc=1.0, s=4, tq=20, mq=7, hq=8, hkv=2, d=64, bs=16, nb=64, mb=8, scale=0.125, window=0, sinks=0)
    a.update(k)
    return t._load().tvl_diff_attention_prefill(*a.values(), None)


@pytest.mark.parametrize("bad,want", [
    (dict(s=-1), "INVALID_ARG"), (dict(tq=-1), "INVALID_ARG"), (dict(mq=-1), "INVALID_ARG"),
    (dict(mq=0), "INVALID_ARG"), (dict(d=128), "UNSUPPORTED"), (dict(bs=24), "UNSUPPORTED"),
    (dict(hq=9), "INVALID_ARG"), (dict(hq=9, hkv=3), "INVALID_ARG"), (dict(hq=18, hkv=2), "UNSUPPORTED"),
    (dict(nb=0), "INVALID_ARG"), (dict(nb=1 << 27), "UNSUPPORTED"), (dict(mb=1 << 26), "UNSUPPORTED"),
    (dict(s=65536), "UNSUPPORTED"), (dict(s=65535, mq=1 << 20), "UNSUPPORTED"),
    (dict(mq=2 ** 31 - 1, s=20), "UNSUPPORTED"), (dict(window=-1), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"),
    (dict(scale=float("inf")), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(out=D16 + 8), "INVALID_ARG"),
    (dict(qsl=None), "INVALID_ARG"), (dict(kc=D16 + 8), "INVALID_ARG"), (dict(lam=None), "INVALID_ARG"),
    (dict(w=D16 + 2), "INVALID_ARG"), (dict(eps=-0.5), "INVALID_ARG"), (dict(osc=float("nan")), "INVALID_ARG")])
def test_prefill_refusals(tvl, bad, want):
    assert _prefill(tvl, **bad) == getattr(tvl, "ERR_" + want)
    assert tvl._load().tvl_last_error()


def test_no_sequences_is_ok(tvl):
    assert _decode(tvl, s=0, out=None, q=None, ws=None) == tvl.OK
    assert _prefill(tvl, s=0, out=None) == tvl.OK and _prefill(tvl, tq=0, mq=0, q=None) == tvl.OK


def test_binding_checks(tvl):
    kv = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tvl.diff_attention_decode(torch.zeros(1, 1, 128), torch.zeros(1, 2, 64), kv, kv, i32.view(1, 1), i32,
                                  torch.zeros(1), 0.125)
    with pytest.raises(ValueError, match="32 bits"):
        tvl.diff_attention_decode(None, None, kv, kv, None, None, None, 0.125, window=2 ** 31)


def test_sizes_past_32_bits_are_refused(tvl):
    with pytest.raises(ValueError, match="32 bits"):
        tvl._c_int(2 ** 31, "max_q_len")
    assert tvl._c_int(7, "x") == 7


def test_plain_form():
    """One key: both maps are its value; equal keys: the mean of the values."""
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 64)), rng.standard_normal((2, 1, 64)), rng.standard_normal((1, 128))
    y, _ = F.pair_row(q[0], q[1], k[0], k[1], v, 0.3, 0.25, None, 0.0, 1.0, 15)
    assert np.allclose(y, 0.75 * v[0], rtol=1e-12)
    v = rng.standard_normal((7, 128))
    y, _ = F.pair_row(q[0], q[1], np.ones((7, 64)), np.ones((7, 64)), v, 0.3, 0.25, np.ones(128), 0.0, 2.0, 15)
    m = v.mean(0)
    assert np.allclose(y, 2 * m / np.sqrt((m * m).mean()), rtol=1e-12)
