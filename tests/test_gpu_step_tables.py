"""Step tables against a plain row-by-row form; every array has to be equal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_198_gb300 as tvl
from gpu_common import DEV, assert_clean_status

pytestmark = pytest.mark.gpu


class Plain:
    """The definition on the host: a stack, and rows one after the other."""

    def __init__(self, tables, free, count, bs):
        self.tables, self.free, self.count, self.bs = tables.copy(), free.copy(), count, bs

    def step(self, cached, new, room):
        bs = self.bs
        lens = list(cached)
        for s, n in enumerate(new):
            if n < 0:
                b = -(-lens[s] // bs)
                self.free[self.count:self.count + b] = self.tables[s, :b]
                self.count += b
                lens[s] = 0
        qsl, slots, pos = [0], [], []
        for s, n in enumerate(new):
            for p in range(lens[s], lens[s] + max(n, 0)):
                if p % bs == 0:
                    self.count -= 1
                    self.tables[s, p // bs] = self.free[self.count]
                slots.append(self.tables[s, p // bs] * bs + p % bs)
                pos.append(p)
            lens[s] += max(n, 0)
            qsl.append(len(slots))
        pad = room - len(slots)
        return lens, qsl, slots + [-1] * pad, pos + [0] * pad


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _state(rng, cached, new, bs, spare=3, width=2):
    blocks = [-(-c // bs) for c in cached]
    need = sum(-(-(c + n) // bs) - b for c, n, b in zip(cached, new, blocks) if n > 0)
    used = sum(blocks)
    nb = used + max(need, 0) + spare
    perm = rng.permutation(nb).astype(np.int32)
    mb = max([1] + [-(-(c + max(n, 0)) // bs) for c, n in zip(cached, new)]) + width
    tables = np.full((len(cached), mb), -7, np.int32)
    at = 0
    for s, n in enumerate(blocks):
        tables[s, :n] = perm[at:at + n]
        at += n
    free = np.full(nb, -9, np.int32)
    free[:nb - used] = perm[used:]
    return tables, free, nb - used


def _call(tables, free, count, cached, new, room, bs, in_place, positions=True):
    """Returns (tables, free, count, context_lens, qsl, slots, positions) on the host."""
    t, f, c, n = _i32(tables), _i32(free), _i32([count]), _i32(new)
    lens = _i32(cached)
    s = len(cached)
    ctx = lens if in_place else torch.full((s,), -5, dtype=torch.int32, device=DEV)
    out = None if in_place else torch.full((1,), -5, dtype=torch.int32, device=DEV)
    qsl = torch.full((s + 1,), -5, dtype=torch.int32, device=DEV)
    slots = torch.full((room,), -5, dtype=torch.int32, device=DEV)
    pos = torch.full((room,), -5, dtype=torch.int32, device=DEV) if positions else None
    tvl.build_step_tables(t, f, ctx, qsl, slots, pos, c, lens, n, bs, free_count_out=out)
    got = [t, f, c if in_place else out, ctx, qsl, slots, pos]
    return [None if x is None else x.cpu().numpy() for x in got]


def _check(seed, cached, new, bs, room=None, in_place=False, positions=True):
    rng = np.random.default_rng(seed)
    tables, free, count = _state(rng, cached, new, bs)
    room = sum(max(n, 0) for n in new) + 5 if room is None else room
    want = Plain(tables, free, count, bs)
    lens, qsl, slots, pos = want.step(cached, new, room)
    got = _call(tables, free, count, cached, new, room, bs, in_place, positions)
    for g, w in zip(got, (want.tables, want.free, [want.count], lens, qsl, slots, pos)):
        if g is not None:
            assert np.array_equal(g, np.asarray(w))
    assert_clean_status()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([17], [-1]), ([0], [-1]), ([0, 0, 0], [0, 0, 0]),
    ([5, 16, 0, 31, 32, 33, 7], [1, 1, 100, 0, -1, -1, 27]), ([100, 3], [-1, 200]),
    ([0, 50, 0, 50], [0, -1, 0, 0]), ([16] * 40, [1] * 40), ([1] * 33, [-1] * 33)])
def test_small_batches(cached, new, in_place):
    _check(1, cached, new, 16, in_place=in_place)


@pytest.mark.parametrize("bs", [1, 3, 16, 32, 64, 128, 1000])
def test_block_sizes(bs):
    _check(2, [0, 1, bs - 1, bs, bs + 1, 5 * bs, 7], [3 * bs, 1, 1, 1, 0, -1, 2 * bs + 1], bs)


@pytest.mark.parametrize("rows", [1, 31, 1000, 1024, 1025, 5000])
def test_many_rows(rows):
    """One CTA's rows and several rounds of them, in one launch and in two."""
    rng = np.random.default_rng(rows)
    cached = [int(x) for x in rng.integers(0, 200, rows)]
    new = [int(x) for x in rng.integers(-1, 3, rows)]
    _check(3, cached, new, 16, in_place=bool(rows & 1))


@pytest.mark.parametrize("tokens", [4090, 4091, 4096, 4097, 30000])
def test_many_tokens(tokens):
    """Both sides of the step's one and two launches."""
    _check(4, [100, 0, 0, 7], [tokens - 50, 0, 20, 30], 16)
    _check(5, [0], [tokens], 32, room=tokens, in_place=True, positions=False)


@pytest.mark.parametrize("seed", range(8))
def test_drawn(seed):
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(1, 300))
    cached = [int(x) for x in rng.integers(0, 900, n)]
    new = [int(x) for x in np.where(rng.random(n) < 0.2, -1, rng.integers(0, 120, n))]
    _check(seed, cached, new, int(rng.choice([8, 16, 48, 128])), in_place=bool(seed & 1))


@pytest.mark.parametrize("room", [10, 5000])
@pytest.mark.parametrize("what,bit", [
    ("negative", tvl.DEV_BAD_CONTEXT_LEN), ("past the table", tvl.DEV_BAD_CONTEXT_LEN),
    ("grows past the table", tvl.DEV_BAD_CONTEXT_LEN), ("tokens", tvl.DEV_BAD_QUERY_LEN),
    ("blocks", tvl.DEV_OUT_OF_BLOCKS), ("count low", tvl.DEV_BAD_BLOCK_ID),
    ("count high", tvl.DEV_BAD_BLOCK_ID), ("given twice", tvl.DEV_BAD_BLOCK_ID)])
def test_refused_steps_change_nothing(what, bit, room):
    rng = np.random.default_rng(9)
    cached, new = [20, 40, 3], [2, -1, 4]
    tables, free, count = _state(rng, cached, new, 16)
    if what == "negative":
        cached = [20, -40, 3]
    elif what == "past the table":
        cached = [20, 40, 16 * tables.shape[1] + 1]
    elif what == "grows past the table":
        new = [2, -1, 2147483647]
    elif what == "tokens":
        new = [2, -1, room - 1]
        tables = np.concatenate([tables, np.full((3, room // 16 + 2), -7, np.int32)], 1)
        free, count = np.concatenate([free, np.arange(400, dtype=np.int32)]), count
    elif what == "blocks":
        new, count = [13, 0, 0], 0
    elif what == "count low":
        count = -1
    elif what == "count high":
        count = len(free) + 1
    else:
        count = len(free) - 1
    for in_place in (False, True):
        got = _call(tables, free, count, cached, new, room, 16, in_place)
        for g, w in zip(got, (tables, free, [count], cached, [0] * 4, [-1] * room, [0] * room)):
            assert np.array_equal(g, np.asarray(w))
        # every reason that holds is reported
        if what == "tokens" and -(-(3 + room - 1) // 16) - 1 > count + 3:
            bit = bit | tvl.DEV_OUT_OF_BLOCKS
        if what == "blocks" and room < 13:
            bit = bit | tvl.DEV_BAD_QUERY_LEN
        assert tvl.get_device_status() == bit


def test_bad_block_ids_are_reported_and_their_slots_skipped():
    tables = np.array([[99, -1, -1], [2, -1, -1]], np.int32)    # 99: the partly filled block
    free = np.array([0, 3, 77, 1], np.int32)
    got = _call(tables, free, 3, [5, 16], [2, 20], 30, 16, False)
    assert got[5].tolist() == [-1] * 2 + [-1] * 16 + [3 * 16 + i for i in range(4)] + [-1] * 8
    assert got[0][1].tolist() == [2, 77, 3] and got[2].tolist() == [1]
    assert tvl.get_device_status() == tvl.DEV_BAD_BLOCK_ID


def test_the_last_slot_of_the_largest_pool():
    """Slots up to 2^31 - 1, through table entries alone."""
    bs, nb = 1 << 20, 2047
    free = np.full(nb, -9, np.int32)
    free[:2] = [5, 2046]
    got = _call(np.full((1, 2), -7, np.int32), free, 2, [0], [bs + 1], bs + 1, bs, False)
    assert got[5][0] == 2046 * bs and got[5][bs - 1] == 2047 * bs - 1 and got[5][bs] == 5 * bs
    assert got[3].tolist() == [bs + 1] and got[2].tolist() == [0]
    assert_clean_status()


def test_a_captured_loop_of_steps():
    """Decode steps in a graph that updates its own lengths, count and tables."""
    rng = np.random.default_rng(11)
    cached, new = [14, 0, 31, 16], [1, 1, 1, 1]
    tables, free, count = _state(rng, cached, [40] * 4, 16, spare=0)
    t, f, c, lens, n = _i32(tables), _i32(free), _i32([count]), _i32(cached), _i32(new)
    qsl, slots, pos = (torch.zeros(k, dtype=torch.int32, device=DEV) for k in (5, 8, 8))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tvl.build_step_tables(t, f, lens, qsl, slots, pos, c, lens, n, 16)
    want = Plain(tables, free, count, 16)
    for step in range(40):
        if step == 20:                     # a row leaves and its place is taken by a new one
            new = [1, -1, 1, 1]
        elif step == 21:
            new = [1, 1, 1, 1]
        n.copy_(_i32(new))
        g.replay()
        cached, wq, ws, wp = want.step(cached, new, 8)
        assert lens.tolist() == cached and qsl.tolist() == wq
        assert slots.tolist() == ws and pos.tolist() == wp
        assert c.tolist() == [want.count] and np.array_equal(t.cpu().numpy(), want.tables)
    assert_clean_status()


def test_another_stream_and_no_rows():
    s = torch.cuda.Stream()
    got = {}
    for stream in (None, s, s.cuda_stream):
        t, f, c = _i32(np.full((2, 4), -7)), _i32([4, 3, 2, 1, 0]), _i32([5])
        ctx, qsl, slots = (torch.full((k,), -5, dtype=torch.int32, device=DEV) for k in (2, 3, 64))
        torch.cuda.synchronize()
        tvl.build_step_tables(t, f, ctx, qsl, slots, None, c, _i32([0, 0]), _i32([17, 3]), 16, stream=stream)
        torch.cuda.synchronize()
        got[str(stream)] = [x.tolist() for x in (t, c, ctx, qsl, slots)]
    assert len({str(v) for v in got.values()}) == 1
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    qsl, slots, c = _i32([-5]), _i32([7, 7]), _i32([1])
    tvl.build_step_tables(e.view(0, 3), _i32([0]), e, qsl, slots, None, c, e, e, 16)
    assert qsl.tolist() == [0] and slots.tolist() == [-1, -1] and c.tolist() == [1]
    assert_clean_status()
