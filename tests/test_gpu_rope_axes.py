"""The paged write with rotary positions of several axes, against the formula in
64 bits.

Bound: a result is the exact rotation rounded to bf16 (2^-8 of it) after an fp32
rotation whose cosine and sine are off by at most 2^-21 (the angle in units of
2^-62 turns is off by position * 2^-53 of a radian at most, 2^-22 at 2^31; its
rounding to fp32 and sincospif's error are below 2^-22 together), two products and
a sum of fp32: 2^-20 (|x_i| + |x_{i+32}|) in all."""
import numpy as np
import pytest
import torch

import paged_kv_cache_198_gb300 as tvl
import window_common as C
from gpu_common import DEV, assert_clean_status, bits_of

pytestmark = pytest.mark.gpu

THETA = 500000.0


def axis_of(sections, interleaved):
    a = len(sections)
    if interleaved:
        return [i % a if i < a * sections[i % a] else 0 for i in range(32)]
    return [j for j, n in enumerate(sections) for _ in range(n)]


def rotated(x, positions, sections, interleaved, theta=THETA):
    """x [T, H, 64] in float64 -> the rotation and its fp32 error bound."""
    axis = axis_of(sections, interleaved)
    assert [axis.count(j) for j in range(len(sections))] == list(sections)
    f = np.float64(np.float32(theta)) ** (-np.arange(32) / 32.0)
    a = (positions[axis].T.astype(np.float64) * f)[:, None]
    x0, x1 = x[..., :32], x[..., 32:]
    out = np.concatenate([x0 * np.cos(a) - x1 * np.sin(a), x1 * np.cos(a) + x0 * np.sin(a)], -1)
    slack = np.tile((np.abs(x0) + np.abs(x1)) * 2.0 ** -20, 2)
    return out, slack


def near(got, want, slack):
    assert (np.abs(got - want) <= (np.abs(want) + slack) * 2.0 ** -8 + slack + 2.0 ** -133).all()


def _bf(rng, shape, spread=1.0):
    return C.bf16_to_f64(C.f64_to_bf16_bits(rng.standard_normal(shape) * spread))


def _slots(rng, t, nb, bs, skip=0.2):
    s = rng.permutation(nb * bs)[:t].astype(np.int32)
    s[rng.random(t) < skip] = -3
    return s


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


AXES = [((32,), False), ((8, 12, 12), False), ((12, 10, 10), True), ((16, 16), False), ((16, 16), True),
        ((2, 10, 10, 10), False), ((8, 8, 8, 8), True), ((11, 11, 10), True), ((30, 1, 1), False)]


def _run(seed, t, hq, hkv, bs, sections, interleaved, top=4000, theta=THETA, spread=1.0, positions=None):
    rng = np.random.default_rng(seed)
    nb = -(-t // bs) + 2
    if positions is None:
        positions = rng.integers(0, top, (len(sections), t)).astype(np.int32)
    q, k, v = (_bf(rng, (t, h, 64), spread) for h in (hq, hkv, hkv))
    old = _bf(rng, (2, nb, bs, hkv, 64))
    slots = _slots(rng, t, nb, bs)
    tq = C.bf16(q, DEV) if hq else None
    kc, vc = C.bf16(old[0], DEV), C.bf16(old[1], DEV)
    tvl.rope_axes_paged_kv_write(tq, C.bf16(k, DEV), C.bf16(v, DEV), kc, vc, _i32(slots), _i32(positions),
                                 sections, interleaved=interleaved, rope_theta=theta)
    if hq:
        near(C.f64(tq), *rotated(q, positions, sections, interleaved, theta))
    want, slack = rotated(k, positions, sections, interleaved, theta)
    new = C.f64(kc).reshape(nb * bs, hkv, 64)
    live = slots >= 0
    near(new[slots[live]], want[live], slack[live])
    wv, wk = old[1].reshape(nb * bs, hkv, 64).copy(), old[0].reshape(nb * bs, hkv, 64)
    wv[slots[live]] = v[live]
    assert np.array_equal(C.f64(vc).reshape(wv.shape), wv)
    other = np.ones(nb * bs, bool)
    other[slots[live]] = False
    assert np.array_equal(new[other], wk[other])
    assert_clean_status()


@pytest.mark.parametrize("sections,interleaved", AXES)
def test_axes(sections, interleaved):
    _run(1, 37, 8, 2, 16, sections, interleaved)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (1, 1), (0, 8), (5, 3), (17, 5), (16, 16), (64, 8), (7, 9), (24, 12)])
def test_heads(hq, hkv):
    _run(2, 13, hq, hkv, 32, (8, 12, 12), False)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 127, 700])
def test_tokens(t):
    _run(3, t, 8, 4, 128, (12, 10, 10), True)


@pytest.mark.parametrize("bs", [1, 7, 16, 64])
def test_block_sizes(bs):
    _run(4, 29, 4, 2, bs, (16, 16), False)


@pytest.mark.parametrize("theta", [1.0625, 10000.0, 1e7])
@pytest.mark.parametrize("spread", [1e-30, 1.0, 1e30])
def test_magnitudes(theta, spread):
    _run(5, 20, 4, 2, 16, (8, 12, 12), False, theta=theta, spread=spread)


def test_far_and_negative_positions():
    p = np.array([[2 ** 31 - 1, -2 ** 31, -1, 0, 1 << 30], [0, 5, -77, 2 ** 31 - 7, 3],
                  [-2 ** 31, 1, 2 ** 31 - 1, -4, 0]], np.int32)
    _run(6, 5, 4, 2, 16, (8, 12, 12), False, positions=p)


def test_text_tokens_equal_the_one_axis_write():
    """The same position on every axis is the plain rotary embedding: the 4-bit
    write bit for bit, and one axis of 32 pairs the same bits as three."""
    rng = np.random.default_rng(7)
    pos = rng.integers(0, 9000, 50)
    q, k, v = (C.bf16(_bf(rng, (50, h, 64)), DEV) for h in (8, 2, 2))
    slots = _i32(rng.permutation(64)[:50])
    bits = []
    for sections, inter in (((32,), False), ((8, 12, 12), False), ((12, 10, 10), True)):
        tq, kc, vc = q.clone(), torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV), \
            torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
        tvl.rope_axes_paged_kv_write(tq, k, v, kc, vc, slots, _i32(np.tile(pos, (len(sections), 1))), sections,
                                     interleaved=inter)
        bits.append([bits_of(x) for x in (tq, kc, vc)])
    for other in bits[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(bits[0], other))
    one, many = (torch.zeros(tvl.kv4_cache_shape(4, 2, 16), dtype=torch.uint8, device=DEV) for _ in range(2))
    q1, q2 = q.clone(), q.clone()
    tvl.kv4_write(k, v, one, slots, q=q1, positions=_i32(pos))
    tvl.kv4_axes_write(k, v, many, slots, q2, _i32(np.tile(pos, (3, 1))), (8, 12, 12))
    assert torch.equal(one, many) and torch.equal(q1, q2)
    assert np.array_equal(bits_of(q1), bits[0][0])
    assert_clean_status()


@pytest.mark.parametrize("sections,interleaved", AXES)
def test_4_bit_write_quantises_the_rotated_rows(sections, interleaved):
    """Codes, scales and offsets of the 4-bit write are those of kv4_write without
    positions on the K rows that the bf16 write stores."""
    rng = np.random.default_rng(8)
    t, hq, hkv, bs = 45, 6, 3, 32
    pos = _i32(rng.integers(-50, 4000, (len(sections), t)))
    q, k, v = (C.bf16(_bf(rng, (t, h, 64)), DEV) for h in (hq, hkv, hkv))
    slots = _slots(rng, t, 3, bs)
    kc, vc = (torch.zeros(3, bs, hkv, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q1, q2 = q.clone(), q.clone()
    tvl.rope_axes_paged_kv_write(q1, k, v, kc, vc, _i32(slots), pos, sections, interleaved=interleaved)
    live = slots >= 0
    rows = kc.view(-1, hkv, 64)[torch.from_numpy(slots[live].astype(np.int64)).to(DEV)].contiguous()
    a, b = (torch.zeros(tvl.kv4_cache_shape(3, hkv, bs), dtype=torch.uint8, device=DEV) for _ in range(2))
    tvl.kv4_write(rows, v[torch.from_numpy(live).to(DEV)].contiguous(), a, _i32(slots[live]))
    tvl.kv4_axes_write(k, v, b, _i32(slots), q2, pos, sections, interleaved=interleaved)
    assert torch.equal(a, b) and torch.equal(q1, q2)
    assert_clean_status()


def test_bad_slots_are_skipped_and_reported():
    rng = np.random.default_rng(9)
    k = C.bf16(_bf(rng, (4, 2, 64)), DEV)
    for four in (False, True):
        kc, vc = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        cache = torch.zeros(tvl.kv4_cache_shape(2, 2, 16), dtype=torch.uint8, device=DEV)
        slots, pos = _i32([3, 32, -1, 2 ** 31 - 1]), _i32(np.zeros((2, 4)))
        if four:
            tvl.kv4_axes_write(k, k, cache, slots, None, pos, (16, 16))
        else:
            tvl.rope_axes_paged_kv_write(None, k, k, kc, vc, slots, pos, (16, 16))
            assert torch.equal(kc.view(-1, 2, 64)[3], k[0]) and int((kc != 0).any(-1).any(-1).sum()) == 1
        assert tvl.get_device_status() == tvl.DEV_BAD_SLOT


def test_refusals():
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots, pos = _i32([0, 1, 2, 3]), _i32(np.zeros((3, 4)))
    for bad in (dict(sections=(16, 16)), dict(sections=(8, 12, 13)), dict(sections=(8, 12, 12), interleaved=True),
                dict(sections=(0, 16, 16)), dict(sections=()), dict(sections=(32,))):
        with pytest.raises((ValueError, tvl.TvlError)):
            tvl.rope_axes_paged_kv_write(None, k, k, kc, kc.clone(), slots, pos, **bad)
    with pytest.raises(ValueError):
        tvl.rope_axes_paged_kv_write(None, k, k, kc, kc.clone(), slots, pos[0], (32,))
    with pytest.raises(ValueError, match="contiguous"):
        tvl.rope_axes_paged_kv_write(None, k, k, kc, kc.clone(), slots, _i32(np.zeros((4, 3))).T, (8, 12, 12))
    with pytest.raises(ValueError):
        tvl.rope_axes_paged_kv_write(None, k, k[:3], kc, kc.clone(), slots, pos, (8, 12, 12))
    assert_clean_status()


def test_captured_and_replayed_with_new_inputs():
    rng = np.random.default_rng(10)
    q, k, v = (C.bf16(_bf(rng, (6, h, 64)), DEV) for h in (4, 2, 2))
    kc, vc = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots, pos = _i32(np.arange(6)), _i32(rng.integers(0, 99, (3, 6)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        tvl.rope_axes_paged_kv_write(q, k, v, kc, vc, slots, pos, (8, 12, 12))
    for _ in range(3):
        x = _bf(rng, (6, 4, 64))
        p = rng.integers(0, 5000, (3, 6)).astype(np.int32)
        q.copy_(C.bf16(x, DEV))
        pos.copy_(_i32(p))
        g.replay()
        near(C.f64(q), *rotated(x, p, (8, 12, 12), False))
    assert_clean_status()
