"""Step tables and rotary positions with several axes without a GPU: refusals of
the C ABI (before any CUDA call) and of the binding."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def tvl():
    from paged_kv_cache_198_gb300 import _build

    _build.build()
    import paged_kv_cache_198_gb300 as t

    return t


def _addr(i):
    """Well separated stand-ins for device pointers; never read."""
    return (i + 1) << 32


NAMES = ("tables", "free", "count_out", "ctx", "qsl", "slots", "pos", "count", "cached", "new")


def _tables(t, **k):
    a = {n: _addr(i) for i, n in enumerate(NAMES)}
    a.update(s=4, n=64, bs=16, nb=32, mb=8)
    a.update(k)
    return t._load().tvl_build_step_tables(*(a[n] for n in NAMES), a["s"], a["n"], a["bs"], a["nb"],
                                           a["mb"], None)


@pytest.mark.parametrize("bad,want", [
    (dict(s=-1), "INVALID_ARG"), (dict(n=-1), "INVALID_ARG"), (dict(bs=0), "INVALID_ARG"),
    (dict(nb=0), "INVALID_ARG"), (dict(mb=0), "INVALID_ARG"),
    (dict(nb=1 << 27, bs=16), "UNSUPPORTED"), (dict(mb=1 << 27, bs=16), "UNSUPPORTED"),
    (dict(tables=None), "INVALID_ARG"), (dict(free=None), "INVALID_ARG"),
    (dict(count=None), "INVALID_ARG"), (dict(count_out=None), "INVALID_ARG"),
    (dict(ctx=None), "INVALID_ARG"), (dict(qsl=None), "INVALID_ARG"),
    (dict(slots=None), "INVALID_ARG"), (dict(cached=None), "INVALID_ARG"),
    (dict(new=None), "INVALID_ARG"), (dict(slots=_addr(5) + 2), "INVALID_ARG"),
    (dict(pos=_addr(5)), "INVALID_ARG"), (dict(pos=_addr(5) + 252), "INVALID_ARG"),
    (dict(new=_addr(3)), "INVALID_ARG"), (dict(ctx=_addr(8) + 4), "INVALID_ARG"),
    (dict(count=_addr(1) + 124), "INVALID_ARG"), (dict(qsl=_addr(3) + 12), "INVALID_ARG"),
    (dict(cached=_addr(0) + 4 * 31), "INVALID_ARG")])
def test_tables_refusals(tvl, bad, want):
    assert _tables(tvl, **bad) == getattr(tvl, "ERR_" + want)
    assert tvl._load().tvl_last_error()


def _axes(t, four, **k):
    a = dict(q=256, k=256, v=256, kc=256, vc=256, slots=256, pos=256, sec=(8, 12, 12), axes=None,
             inter=0, n=4, hq=4, hkv=2, d=64, bs=16, nb=8, theta=10000.0)
    a.update(k)
    sec = a["sec"] and (ctypes.c_int * len(a["sec"]))(*a["sec"])
    axes = len(a["sec"] or ()) if a["axes"] is None else a["axes"]
    tail = (a["slots"], a["pos"], sec, axes, a["inter"], a["n"], a["hq"], a["hkv"], a["d"], a["bs"],
            a["nb"], a["theta"], None)
    if four:
        return t._load().tvl_kv4_axes_write(a["q"], a["k"], a["v"], a["kc"], *tail)
    return t._load().tvl_rope_axes_paged_kv_write(a["q"], a["k"], a["v"], a["kc"], a["vc"], *tail)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("bad,want", [
    (dict(d=128), "UNSUPPORTED"), (dict(n=-1), "INVALID_ARG"), (dict(hkv=0), "INVALID_ARG"),
    (dict(nb=0), "INVALID_ARG"), (dict(kc=None), "INVALID_ARG"), (dict(kc=264), "INVALID_ARG"),
    (dict(k=None), "INVALID_ARG"), (dict(v=258), "INVALID_ARG"), (dict(q=260), "INVALID_ARG"),
    (dict(hq=0), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"),
    (dict(theta=1.0), "INVALID_ARG"), (dict(theta=float("inf")), "INVALID_ARG"),
    (dict(hq=524281), "UNSUPPORTED"), (dict(hkv=262137), "UNSUPPORTED"),
    (dict(sec=None, axes=3), "INVALID_ARG"), (dict(axes=0), "UNSUPPORTED"),
    (dict(sec=(7, 7, 6, 6, 6)), "UNSUPPORTED"), (dict(sec=(16, 15)), "INVALID_ARG"),
    (dict(sec=(32, 0)), "INVALID_ARG"), (dict(sec=(40, -8)), "INVALID_ARG"),
    (dict(sec=(8, 12, 12), inter=1), "INVALID_ARG"), (dict(sec=(15, 17), inter=1), "INVALID_ARG")])
def test_axes_refusals(tvl, four, bad, want):
    assert _axes(tvl, four, **bad) == getattr(tvl, "ERR_" + want)
    assert tvl._load().tvl_last_error()


@pytest.mark.parametrize("four", [False, True])
def test_no_tokens_is_ok(tvl, four):
    assert _axes(tvl, four, n=0, k=None, v=None, slots=None, pos=None) == tvl.OK


def test_binding_checks(tvl):
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tvl.build_step_tables(i32.view(2, 2), i32, i32, i32, i32, i32, i32, i32, i32, 16)
    with pytest.raises(TypeError):
        tvl.build_step_tables(i32.view(2, 2).long(), i32, i32, i32, i32, i32, i32, i32, i32, 16)
    kv = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tvl.rope_axes_paged_kv_write(None, kv[0], kv[0], kv, kv, i32, i32.view(1, 4), [32])
    with pytest.raises(ValueError, match="CUDA"):
        tvl.kv4_axes_write(kv[0], kv[0], torch.zeros(2, 1, 2, 1152, dtype=torch.uint8), i32, None,
                           i32.view(1, 4), [32])


def test_more_rows_than_the_loops_count_are_refused(tvl):
    assert _tables(tvl, s=(1 << 30) + 1, mb=1) == tvl.ERR_UNSUPPORTED
