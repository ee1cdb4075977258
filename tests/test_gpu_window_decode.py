"""Decode attention with a sliding window and sinks over the bf16 caches,
against the plain form in 64 bits (tests/window_common.py derives the bounds)."""
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


def _run(seed, ctx, hq, hkv, bs, window, sinks, spread=1.0, poison=False, scale=0.125):
    rng = np.random.default_rng(seed)
    tables, nb = C.deal(rng, ctx, bs)
    k, v = _bf(rng, (nb, bs, hkv, 64), spread), _bf(rng, (nb, bs, hkv, 64), spread)
    q = _bf(rng, (len(ctx), hq, 64), 1.5)
    want, tol = C.decode_ref(q, tables, ctx, scale, window, sinks, kv=(k, v))
    if poison:                      # every slot that is not visible, and the unread table entries
        seen = np.zeros((nb, bs), bool)
        for s, n in enumerate(ctx):
            if n:
                p = C.visible(n - 1, window, sinks)
                seen[tables[s][p // bs], p % bs] = True
                keep = np.zeros(tables.shape[1], bool)
                keep[p // bs] = True
                tables[s][~keep] = -12345
        k[~seen], v[~seen] = np.nan, np.inf
    out = torch.full(q.shape, float("nan"), device=DEV)
    tvl.paged_attention_window_decode(out, C.bf16(q, DEV), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables),
                                      _cuda(np.asarray(ctx, np.int32)), scale, window, sinks=sinks)
    got = C.f64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv,bs", [
    (8, 2, 16), (32, 8, 16), (8, 8, 32), (64, 8, 32), (5, 5, 64), (6, 1, 128), (21, 3, 16),
    (24, 12, 32), (14, 7, 16), (16, 16, 64), (8, 1, 16), (40, 8, 16)])
def test_heads(hq, hkv, bs):
    _run(20 + hq, [1, 700, 16, 17, 333], hq, hkv, bs, 200, 5)


@pytest.mark.parametrize("ctx", [[1], [15], [16], [31, 33], [0, 5, 0], [0], [2000], [64] * 40,
                                 list(range(1, 200, 3)), [7] * 700])
def test_lengths(ctx):
    _run(40, ctx, 8, 2, 16, 100, 4)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 7), (1, 0), (1, 1), (16, 0), (17, 4), (100, 16),
                                          (100, 17), (64, 1000), (5000, 4), (640, 300)])
@pytest.mark.parametrize("bs", [16, 64])
def test_windows_with_poisoned_unseen_slots(window, sinks, bs):
    _run(50, [1, 90, 0, 101, 1500, 640, 116], 12, 3, bs, window, sinks, poison=True)


@pytest.mark.parametrize("spread", [1e-6, 1e4])
def test_magnitudes(spread):
    _run(60, [500, 77], 16, 4, 16, 300, 4, spread=spread)


def test_window_of_the_whole_context_equals_the_plain_decode():
    """Against paged_attention_decode on the same inputs, within both bounds."""
    rng = np.random.default_rng(70)
    ctx = [900, 3, 0, 1777]
    tables, nb = C.deal(rng, ctx, 16)
    k, v, q = (_bf(rng, s) for s in ((nb, 16, 8, 64), (nb, 16, 8, 64), (4, 32, 64)))
    args = [C.bf16(q, DEV), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables), _cuda(np.asarray(ctx, np.int32)), 0.125]
    a, b, c = (torch.empty(4, 32, 64, device=DEV) for _ in range(3))
    tvl.paged_attention_decode(a, *args)
    tvl.paged_attention_window_decode(b, *args, 0)
    tvl.paged_attention_window_decode(c, *args, 1777)
    _, tol = C.decode_ref(q, tables, ctx, 0.125, 0, 0, kv=(k, v))
    assert (np.abs(C.f64(a) - C.f64(b)) <= 2 * tol).all()
    assert torch.equal(b, c)


def test_repeats_bit_for_bit_and_from_two_graphs_of_one_workspace():
    rng = np.random.default_rng(71)
    ctx = [3, 900, 0, 450, 77]
    tables, nb = C.deal(rng, ctx, 16)
    k, v, q = (C.bf16(_bf(rng, s), DEV) for s in ((nb, 16, 8, 64), (nb, 16, 8, 64), (5, 32, 64)))
    tab, ln = _cuda(tables), _cuda(np.asarray(ctx, np.int32))
    ws = torch.empty(tvl.window_decode_workspace_size(32, 8), dtype=torch.uint8, device=DEV)
    outs = [torch.full((5, 32, 64), float("nan"), device=DEV) for _ in range(4)]
    for i, w in ((0, 128), (1, 500)):
        tvl.paged_attention_window_decode(outs[i], q, k, v, tab, ln, 0.125, w, sinks=2)
    graphs = []
    for i, w in ((2, 128), (3, 500)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tvl.paged_attention_window_decode(outs[i], q, k, v, tab, ln, 0.125, w, sinks=2, workspace=ws)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert_clean_status()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(900 + seed)
    hkv, g = int(rng.integers(1, 17)), int(rng.integers(1, 9))
    n = int(rng.integers(1, 9))
    ctx = [int(x) for x in np.exp(rng.uniform(0, np.log(1500), n))]
    _run(1000 + seed, ctx, hkv * g, hkv, int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 800)),
         int(rng.integers(0, 70)), poison=bool(seed & 1))


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_workspace_of_its_own_on_another_stream(as_handle):
    """Without a workspace the call allocates one; on a stream other than the
    current one its memory must not be handed to the current stream while the
    call's kernels may still run."""
    rng = np.random.default_rng(77)
    ctx = rng.integers(200, 900, 40).astype(np.int32)
    bs, hkv, hq = 16, 8, 32
    need = -(-ctx // bs)
    nb = int(need.sum())
    tables = np.full((len(ctx), int(need.max())), -1, np.int32)
    ids, at = rng.permutation(nb).astype(np.int32), 0
    for i, n in enumerate(need):
        tables[i, :n] = ids[at:at + n]
        at += n
    k, v = (torch.randn(nb, bs, hkv, 64, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(len(ctx), hq, 64, device=DEV, dtype=torch.bfloat16)
    args = (q, k, v, _cuda(tables), _cuda(ctx), 0.125, 0)
    want = torch.empty(len(ctx), hq, 64, device=DEV)
    tvl.paged_attention_window_decode(want, *args)
    size = tvl.window_decode_workspace_size(hq, hkv)
    side = torch.cuda.Stream(DEV)
    outs = [torch.empty_like(want) for _ in range(30)]
    torch.cuda.synchronize()
    for o in outs:
        tvl.paged_attention_window_decode(o, *args, stream=side.cuda_stream if as_handle else side)
        torch.full((size,), 255, dtype=torch.uint8, device=DEV)      # the current stream's memory
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    assert_clean_status()


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
@pytest.mark.parametrize("hq", [8, 16])
def test_scales(scale, hq):
    _run(80, [300, 700] * 60, hq, 2, 16, 200, 4, scale=scale)


@pytest.mark.parametrize("group", range(1, 9))
@pytest.mark.parametrize("ctx,window,sinks", [(2100, 700, 4), (2100, 736, 0), (768, 0, 0), (2100, 512, 200)])
def test_the_longest_sequences_of_few(group, ctx, window, sinks):
    """Few short bounded sequences: around the most chunks that one CTA holds."""
    _run(90 + group, [ctx, 40], group, 1, 16, window, sinks)


def test_a_workspace_for_the_default_stream_given_as_a_handle():
    """The handle of the default stream is 0: the workspace of a call on it belongs to
    that stream, not to one of torch's own."""
    with tvl._stream_context(torch.cuda.default_stream().cuda_stream):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    rng = np.random.default_rng(78)
    tables, nb = C.deal(rng, [300, 90], 16)
    k, v, q = (_bf(rng, s) for s in ((nb, 16, 2, 64), (nb, 16, 2, 64), (2, 8, 64)))
    want, tol = C.decode_ref(q, tables, [300, 90], 0.125, 0, 0, kv=(k, v))
    out = torch.empty(2, 8, 64, device=DEV)
    args = [C.bf16(q, DEV), C.bf16(k, DEV), C.bf16(v, DEV), _cuda(tables), _cuda(np.array([300, 90], np.int32)), 0.125]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream(DEV)):
        tvl.paged_attention_window_decode(out, *args, 0, stream=0)
    torch.cuda.synchronize()
    assert (np.abs(C.f64(out) - want) <= tol).all()
    assert_clean_status()


@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8), (16, 16)])
@pytest.mark.parametrize("n,top,window", [(200, 900, 0), (200, 900, 300), (600, 120, 0)])
def test_more_sequences_than_ctas(hq, hkv, n, top, window):
    """More sequences than CTAs (and than threads of one), whose lengths make most
    CTAs end inside a sequence: one split sequence a CTA in the list to merge."""
    _run(110 + n, [int(x) for x in np.random.default_rng(n).integers(0, top, n)], hq, hkv, 16, window, 3)


@pytest.mark.parametrize("hq,hkv,window", [(2, 2, 300), (8, 1, 3000), (160, 160, 300)])
def test_the_longest_context(hq, hkv, window):
    """A context of 2^31 - 128 tokens, nearly all of them behind the window: the
    result of the same last rows at the end of a short context."""
    bs, short = 128, 128 * 24
    tables, nb = C.deal(np.random.default_rng(3), [short], bs)
    rng = np.random.default_rng(4)
    k, v, q = (_bf(rng, s) for s in ((nb, bs, hkv, 64), (nb, bs, hkv, 64), (1, hq, 64)))
    mb = (2 ** 31 - 128) // bs
    far = torch.full((1, mb), -1, dtype=torch.int32, device=DEV)
    far[0, mb - short // bs:] = _cuda(tables[0])
    out = torch.full((1, hq, 64), float("nan"), device=DEV)
    for cut in (0, 5):
        tvl.paged_attention_window_decode(out, C.bf16(q, DEV), C.bf16(k, DEV), C.bf16(v, DEV), far,
                                          torch.tensor([2 ** 31 - 128 - cut], dtype=torch.int32, device=DEV), 0.125,
                                          window)
        want, tol = C.decode_ref(q, tables, [short - cut], 0.125, window, 0, kv=(k, v))
        assert (np.abs(C.f64(out) - want) <= tol).all(), (np.abs(C.f64(out) - want) / tol).max()
    assert_clean_status()
