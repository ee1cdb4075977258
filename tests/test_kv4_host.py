"""The 4-bit cache and the windowed decode without a GPU: refusals of the C
ABI (before any CUDA call) and of the binding, and the quantiser's definition
in the plain form that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import window_common as C


@pytest.fixture(scope="module")
def tvl():
    from paged_kv_cache_198_gb300 import _build

    _build.build()
    import paged_kv_cache_198_gb300 as t

    return t


D16 = 256      # a well aligned stand-in for a device pointer; never read


def _write(t, **k):
    a = dict(q=None, k=D16, v=D16, cache=D16, slots=D16, pos=None, n=4, hq=0, hkv=2, d=64, bs=16,
             nb=8, theta=10000.0)
    a.update(k)
    return t._load().tvl_kv4_write(a["q"], a["k"], a["v"], a["cache"], a["slots"], a["pos"], a["n"],
                                   a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["theta"], None)


@pytest.mark.parametrize("bad,want", [
    (dict(d=128), "UNSUPPORTED"), (dict(bs=8), "UNSUPPORTED"), (dict(bs=48), "UNSUPPORTED"),
    (dict(n=-1), "INVALID_ARG"), (dict(hkv=0), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"),
    (dict(cache=None), "INVALID_ARG"), (dict(cache=D16 + 8), "INVALID_ARG"),
    (dict(k=None), "INVALID_ARG"), (dict(v=D16 + 2), "INVALID_ARG"),
    (dict(slots=None), "INVALID_ARG"), (dict(q=D16, hq=4), "INVALID_ARG"),
    (dict(q=D16, hq=0, pos=D16), "INVALID_ARG"), (dict(q=D16 + 4, hq=4, pos=D16), "INVALID_ARG"),
    (dict(pos=D16, theta=1.0), "INVALID_ARG"), (dict(pos=D16, theta=float("nan")), "INVALID_ARG"),
    (dict(hq=-1), "INVALID_ARG")])
def test_write_refusals(tvl, bad, want):
    assert _write(tvl, **bad) == getattr(tvl, "ERR_" + want)
    assert tvl._load().tvl_last_error()


def test_write_of_no_tokens_is_ok(tvl):
    assert _write(tvl, n=0, k=None, v=None, slots=None) == tvl.OK


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), "INVALID_ARG"), (dict(d=32), "UNSUPPORTED"), (dict(bs=20), "UNSUPPORTED"),
    (dict(src=None), "INVALID_ARG"), (dict(cache=D16 + 1), "INVALID_ARG"), (dict(ob=0), "INVALID_ARG")])
def test_expand_and_copy_refusals(tvl, bad, want):
    a = dict(kc=D16, vc=D16, cache=D16, src=D16, dst=D16, n=2, hkv=2, d=64, bs=16, nb=8, ob=8)
    a.update(bad)
    lib = tvl._load()
    want = getattr(tvl, "ERR_" + want)
    assert lib.tvl_kv4_expand_blocks(a["kc"], a["vc"], a["cache"], a["src"], a["dst"], a["n"],
                                     a["hkv"], a["d"], a["bs"], a["nb"], a["ob"], None) == want
    if "ob" not in bad:
        assert lib.tvl_kv4_copy_blocks(a["cache"], a["src"], a["dst"], a["n"], a["hkv"], a["d"],
                                       a["bs"], a["nb"], None) == want


def _decode(t, four, **k):
    a = dict(out=D16, q=D16, kc=D16, vc=D16, tab=D16, ctx=D16, s=4, hq=8, hkv=2, d=64, bs=16, nb=64,
             mb=8, scale=0.125, window=32, sinks=4, ws=D16, wsb=1 << 30)
    a.update(k)
    lib = t._load()
    fn = lib.tvl_kv4_attention_decode if four else lib.tvl_paged_attention_window_decode
    caches = (a["kc"],) if four else (a["kc"], a["vc"])
    return fn(a["out"], a["q"], *caches, a["tab"], a["ctx"], a["s"], a["hq"], a["hkv"], a["d"],
              a["bs"], a["nb"], a["mb"], a["scale"], a["window"], a["sinks"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("bad,want", [
    (dict(s=-1), "INVALID_ARG"), (dict(d=128), "UNSUPPORTED"), (dict(bs=24), "UNSUPPORTED"),
    (dict(hq=18), "UNSUPPORTED"), (dict(hq=7), "INVALID_ARG"), (dict(hkv=0), "INVALID_ARG"),
    (dict(mb=0), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"),
    (dict(sinks=-1), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
    (dict(nb=1 << 27, bs=16), "UNSUPPORTED"), (dict(mb=1 << 27, bs=16), "UNSUPPORTED"),
    (dict(out=None), "INVALID_ARG"), (dict(q=D16 + 8), "INVALID_ARG"), (dict(kc=None), "INVALID_ARG"),
    (dict(tab=None), "INVALID_ARG"), (dict(ctx=None), "INVALID_ARG"), (dict(ws=None), "WORKSPACE"),
    (dict(ws=D16 + 4), "INVALID_ARG")])
def test_decode_refusals(tvl, four, bad, want):
    assert _decode(tvl, four, **bad) == getattr(tvl, "ERR_" + want)


@pytest.mark.parametrize("four", [True, False])
def test_decode_of_no_sequences_is_ok(tvl, four):
    assert _decode(tvl, four, s=0, out=None, q=None, tab=None, ctx=None, ws=None, wsb=0) in (
        (tvl.OK, tvl.ERR_INVALID_ARG) if four else (tvl.OK,))


def test_workspace_size_refusals(tvl):
    lib = tvl._load()
    n = ctypes.c_size_t(0)
    assert lib.tvl_window_decode_workspace_size(8, 2, 64, None) == tvl.ERR_INVALID_ARG
    assert lib.tvl_window_decode_workspace_size(9, 1, 64, ctypes.byref(n)) == tvl.ERR_UNSUPPORTED
    assert lib.tvl_window_decode_workspace_size(8, 2, 96, ctypes.byref(n)) == tvl.ERR_UNSUPPORTED


def test_binding_refusals(tvl):
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(tvl.kv4_cache_shape(8, 2, 16), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        tvl.kv4_write(k, k, cache, slots)
    with pytest.raises(TypeError, match="uint8"):
        tvl.kv4_write(k, k, cache.float(), slots)
    with pytest.raises(ValueError):
        tvl.kv4_cache_shape(8, 2, 24)
    assert tvl.kv4_cache_shape(8, 2, 64) == (8, 4, 2, 1152)


def test_plain_quantiser_keeps_every_value_within_half_a_step():
    rng = np.random.default_rng(1)
    x = C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal((50, 64)) * rng.uniform(0.01, 30, (50, 1))))
    x[0] = 1.5
    c, s, z = C.quantise(x)
    assert (c[0] == 0).all() and s[0] == 0 and z[0] == 1.5
    assert (np.abs(c * s[:, None] + z[:, None] - x) <= s[:, None] / 2 * (1 + 1e-12)).all()
    assert np.array_equal(C.bf16_to_f64(C.f64_to_bf16_bits(s)), s)     # s is a bf16 number
    assert (15 * s >= x.max(-1) - z).all()


def test_plain_cache_packs_what_it_unpacks():
    rng = np.random.default_rng(2)
    cache = C.random_cache(rng, 3, 32, 2)
    codes, s, z = C.unpack(cache)
    assert codes.shape == (2, 3, 32, 2, 64) and (s > 0).all()
    # dimension d of token t: byte 32 t + d / 2 of the record, low half first
    b = cache[1, 1, 0, 512 + 32 * 5 + 9]
    assert codes[1, 1, 16 + 5, 0, 18] == (b & 15) and codes[1, 1, 16 + 5, 0, 19] == (b >> 4)


@pytest.mark.parametrize("bad,want", [
    (dict(window=-1), "INVALID_ARG"), (dict(sinks=-2), "INVALID_ARG"), (dict(d=128), "UNSUPPORTED"),
    (dict(bs=24), "UNSUPPORTED"), (dict(hq=6), "UNSUPPORTED"), (dict(mb=1 << 26), "UNSUPPORTED"),
    (dict(out=None), "INVALID_ARG"), (dict(out=D16 + 8), "INVALID_ARG"), (dict(maxq=0), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(s=-1), "INVALID_ARG"), (dict(s=70000), "UNSUPPORTED")])
def test_window_prefill_refusals(tvl, bad, want):
    a = dict(out=D16, q=D16, qsl=D16, kc=D16, vc=D16, tab=D16, ctx=D16, s=2, tq=10, maxq=8, hq=8, hkv=2,
             d=64, bs=16, nb=64, mb=8, scale=0.125, window=32, sinks=4)
    a.update(bad)
    rc = tvl._load().tvl_paged_attention_window_prefill(
        a["out"], a["q"], a["qsl"], a["kc"], a["vc"], a["tab"], a["ctx"], a["s"], a["tq"], a["maxq"], a["hq"],
        a["hkv"], a["d"], a["bs"], a["nb"], a["mb"], a["scale"], a["window"], a["sinks"], None)
    assert rc == getattr(tvl, "ERR_" + want)


def test_sizes_past_the_launch_grid_are_refused(tvl):
    assert _write(tvl, hkv=65536) == tvl.ERR_UNSUPPORTED
    assert _write(tvl, q=D16, pos=D16, hq=524281) == tvl.ERR_UNSUPPORTED
    lib = tvl._load()
    assert lib.tvl_kv4_expand_blocks(D16, D16, D16, D16, D16, 1 << 28, 8, 64, 128, 8, 8,
                                     None) == tvl.ERR_UNSUPPORTED
    assert _decode(tvl, True, hq=262144, hkv=32768) == tvl.ERR_UNSUPPORTED


@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (2 ** 32 + 5, 0), (5, 2 ** 32), (-2 ** 32, 0), (5, -2 ** 31 - 1)])
def test_windows_past_32_bits_are_refused(tvl, window, sinks):
    """ctypes keeps the lower 32 bits of an argument: 2^32 + 5 would be a window of 5."""
    x = torch.zeros(1)                 # no tensor is looked at before the window
    for call in (tvl.kv4_attention_decode, tvl.bind_kv4_attention_decode):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, x, x, x, x, 0.125, window=window, sinks=sinks)
    for call in (tvl.paged_attention_window_decode, tvl.bind_paged_attention_window_decode):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, x, x, x, x, x, 0.125, window, sinks=sinks)
    for call in (tvl.paged_attention_window_prefill, tvl.bind_paged_attention_window_prefill):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, x, x, x, x, x, x, 0.125, 8, window, sinks=sinks)
    assert tvl._visibility(2 ** 31 - 1, 0) == (2 ** 31 - 1, 0) and tvl._visibility(-1, -1) == (-1, -1)
