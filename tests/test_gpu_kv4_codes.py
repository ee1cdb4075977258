"""Codes of the 4-bit write where the quotient's estimate is least exact, and its
q rows where a warp takes two batches of them.  Codes are whole numbers of a
definition in 64 bits, so they are equal; q's rotation is the bf16 write's, bit
for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_198_gb300 as tvl
import window_common as C
from gpu_common import DEV, assert_clean_status

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


@pytest.mark.parametrize("steps", [1, 2, 7, 15, 30, 31, 255, 1000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_of_close_values(steps, sign):
    """Values a few bf16 steps from one another: the largest minimum for a scale,
    ties in most rows.  Differences are exact in fp32."""
    rng = np.random.default_rng(steps)
    t, hkv, bs = 96, 8, 16
    base = rng.integers(0x3e00, 0x4200, (2, t, hkv, 1))
    base[0, :8] = 0x3f80                                  # 1, and the value below 2
    base[0, 8:16] = 0x3fff
    bits = base + rng.integers(0, steps + 1, (2, t, hkv, 64))
    x = sign * (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    slots = rng.permutation(t).astype(np.int32)
    cache = torch.zeros(tvl.kv4_cache_shape(t // bs, hkv, bs), dtype=torch.uint8, device=DEV)
    tvl.kv4_write(C.bf16(x[0], DEV), C.bf16(x[1], DEV), cache, _i32(slots))
    codes, s, z = C.unpack(cache.cpu().numpy())
    for part in range(2):
        c0, s0, z0 = C.quantise(x[part])
        page, off = slots // bs, slots % bs
        assert np.array_equal(z[part][page, off], z0) and np.array_equal(s[part][page, off], s0)
        assert np.array_equal(codes[part][page, off], c0)
    assert_clean_status()


@pytest.mark.parametrize("t,hq", [(2600, 32), (5000, 17), (2200, 40), (1300, 63), (4700, 18), (9000, 16)])
def test_two_batches_of_q_rows(t, hq):
    """q as the bf16 write turns it, and the cache as smaller calls write it."""
    assert t * hq > 80000
    rng = np.random.default_rng(hq)
    hkv, bs, sections = 2, 16, (8, 12, 12)
    nb = -(-t // bs)
    q, k, v = (torch.randn(t, h, 64, device=DEV).to(torch.bfloat16) for h in (hq, hkv, hkv))
    pos = _i32(rng.integers(0, 100000, (3, t)))
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    slots[::11] = -1
    slots = _i32(slots)
    want, got, small = q.clone(), q.clone(), q.clone()
    kc, vc = (torch.zeros(nb, bs, hkv, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tvl.rope_axes_paged_kv_write(want, k, v, kc, vc, slots, pos, sections)
    a, b = (torch.zeros(tvl.kv4_cache_shape(nb, hkv, bs), dtype=torch.uint8, device=DEV) for _ in range(2))
    tvl.kv4_axes_write(k, v, a, slots, got, pos, sections)
    for i in range(0, t, 700):
        j = slice(i, min(i + 700, t))
        tvl.kv4_axes_write(k[j], v[j], b, slots[j], small[j], pos[:, j].contiguous(), sections)
    assert torch.equal(got, want) and torch.equal(small, want) and torch.equal(a, b)
    assert_clean_status()
