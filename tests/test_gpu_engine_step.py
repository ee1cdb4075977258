"""An engine's steps with the calls that go together: tables from request lengths, the
write with positions of several axes, differential prefill and decode -- prompts come
in chunks, rows decode, leave and are followed by others.  The tables are checked
against the plain row-by-row form, the written rows and the attention against the
formulas in 64 bits on the cache's contents."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import diff_common as F
import paged_kv_cache_198_gb300 as tvl
import window_common as C
from gpu_common import DEV, assert_clean_status
from test_gpu_rope_axes import near, rotated
from test_gpu_step_tables import Plain, _i32

pytestmark = pytest.mark.gpu

HQ, HKV, BS, SECTIONS = 8, 4, 16, (8, 12, 12)


class Engine:
    def __init__(self, rows, blocks, width, room, four=False):
        self.rng = np.random.default_rng(5)
        self.rows, self.room, self.four = rows, room, four
        free = self.rng.permutation(blocks).astype(np.int32)
        self.plain = Plain(np.full((rows, width), -7, np.int32), free, blocks, BS)
        self.tables, self.free, self.count = _i32(self.plain.tables), _i32(free), _i32([blocks])
        self.lens, self.new = _i32(np.zeros(rows)), _i32(np.zeros(rows))
        self.qsl, self.slots, self.pos = _i32(np.zeros(rows + 1)), _i32(np.zeros(room)), _i32(np.zeros(room))
        self.axes = torch.zeros(3, room, dtype=torch.int32, device=DEV)
        self.q, self.k, self.v = (torch.zeros(room, h, 64, dtype=torch.bfloat16, device=DEV) for h in (HQ, HKV, HKV))
        self.kc, self.vc = (torch.zeros(blocks, BS, HKV, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.cache = torch.zeros(tvl.kv4_cache_shape(blocks, HKV, BS), dtype=torch.uint8, device=DEV)
        self.lam = torch.from_numpy(self.rng.uniform(0.1, 0.8, HQ // 2).astype(np.float32)).to(DEV)
        self.weight = C.bf16(self.rng.uniform(0.5, 1.5, 128), DEV)
        self.out = torch.zeros(room, HQ // 2, 128, dtype=torch.bfloat16, device=DEV)
        self.cached = [0] * rows

    def bookkeeping(self):
        tvl.build_step_tables(self.tables, self.free, self.lens, self.qsl, self.slots, self.pos, self.count,
                              self.lens, self.new, BS)

    def write(self):
        """q, K and V of the packed (padded) tokens: text, so the same position on every axis."""
        self.axes.copy_(self.pos.expand(3, -1))
        if self.four:
            tvl.kv4_axes_write(self.k, self.v, self.cache, self.slots, self.q, self.axes, SECTIONS)
        else:
            tvl.rope_axes_paged_kv_write(self.q, self.k, self.v, self.kc, self.vc, self.slots, self.axes, SECTIONS)

    def draw(self, new):
        self.new.copy_(_i32(new))
        self.x = [C.bf16_to_f64(C.f64_to_bf16_bits(self.rng.standard_normal((self.room, h, 64)))) for h in (HQ, HKV, HKV)]
        for t, x in zip((self.q, self.k, self.v), self.x):
            t.copy_(C.bf16(x, DEV))

    def check(self, new, prefill, out):
        """The step's arrays, written rows and attention."""
        self.cached, qsl, slots, pos = self.plain.step(self.cached, new, self.room)
        for got, want in ((self.lens, self.cached), (self.qsl, qsl), (self.slots, slots), (self.pos, pos),
                          (self.count, [self.plain.count]), (self.tables, self.plain.tables)):
            assert np.array_equal(got.cpu().numpy(), np.asarray(want))
        n = qsl[-1]
        p3 = np.tile(np.asarray(pos, np.int32), (3, 1))
        near(C.f64(self.q)[:n], *[y[:n] for y in rotated(self.x[0], p3, SECTIONS, False)])
        kc, vc = C.f64(self.kc), C.f64(self.vc)
        at = np.asarray(slots[:n])
        want, slack = rotated(self.x[1], p3, SECTIONS, False)
        near(kc.reshape(-1, HKV, 64)[at], want[:n], slack[:n])
        assert np.array_equal(vc.reshape(-1, HKV, 64)[at], self.x[2][:n])
        live = [s for s in range(self.rows) if new[s] > 0]
        starts = np.concatenate([[0], np.cumsum([new[s] for s in live])])
        want, tol = F.reference(C.f64(self.q)[:n], starts, self.plain.tables[live], [self.cached[s] for s in live], kc,
                                vc, C.f64(self.lam), 0.125, weight=C.f64(self.weight), eps=np.float64(np.float32(1e-5)),
                                out_scale=0.5, bits=11 if prefill else 15, prefill=prefill)
        got = C.f64(out)
        got = got[:n] if prefill else got[live]
        assert (np.abs(got - want) <= tol).all()
        assert_clean_status()


def test_prompts_decode_steps_and_departures():
    e = Engine(rows=5, blocks=60, width=12, room=160)
    for new in ([70, 1, 0, 33, 16], [20, 90, 5, 0, 1], [0, 0, 40, 17, 0]):      # prompts in chunks
        e.draw(new)
        e.bookkeeping()
        e.write()
        e.out.fill_(float("nan"))
        tvl.diff_attention_prefill(e.out, e.q, e.qsl, e.kc, e.vc, e.tables, e.lens, e.lam, 0.125, 128,
                                   norm_weight=e.weight, out_scale=0.5)
        e.check(new, True, e.out)
        assert e.out[int(e.qsl[-1]):].isnan().all()       # rows behind the last sequence are left
    out = torch.zeros(5, HQ // 2, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(5, HQ, 64, dtype=torch.bfloat16, device=DEV)
    for step in range(6):
        new = [1, 1, 1, 1, 1]
        if step == 2:
            new[1] = -1                                   # done: its blocks go back
        if step > 2:
            new[1] = 0 if step == 3 else 1                # an empty place, then a new request's first tokens
        e.draw(new)
        e.bookkeeping()
        e.write()
        rows = [s for s in range(5) if new[s] > 0]
        q.zero_()
        q[rows] = e.q[:len(rows)]                         # packed tokens to their rows
        tvl.diff_attention_decode(out, q, e.kc, e.vc, e.tables, e.lens, e.lam, 0.125, norm_weight=e.weight, out_scale=0.5)
        e.check(new, False, out)
        assert step not in (2, 3) or not out[1].any()     # nothing cached: a zero row


def test_a_captured_decode_loop():
    """Tables, write and decode of one token a row in a graph that keeps its own lengths."""
    e = Engine(rows=3, blocks=40, width=8, room=3)
    out = torch.zeros(3, HQ // 2, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(tvl.diff_decode_workspace_size(HQ, HKV), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.bookkeeping()
        e.write()
        tvl.diff_attention_decode(out, e.q, e.kc, e.vc, e.tables, e.lens, e.lam, 0.125, norm_weight=e.weight,
                                  out_scale=0.5, workspace=ws)
    for _ in range(40):
        e.draw([1, 1, 1])
        g.replay()
        e.check([1, 1, 1], False, out)


def test_the_4_bit_cache_with_the_same_tables():
    """kv4_axes_write into the step's slots is kv4_write of the rows rotated by the bf16 write."""
    e, f = Engine(rows=2, blocks=12, width=4, room=32), Engine(rows=2, blocks=12, width=4, room=32, four=True)
    want = torch.zeros_like(f.cache)
    for new in ([20, 3], [1, 9], [1, -1]):
        for x in (e, f):
            x.draw(new)
            x.bookkeeping()
            x.write()
        live = e.slots >= 0
        at = e.slots[live].long()
        tvl.kv4_write(e.kc.view(-1, HKV, 64)[at].contiguous(), e.vc.view(-1, HKV, 64)[at].contiguous(), want,
                      e.slots[live].contiguous())
        assert torch.equal(f.cache, want) and torch.equal(e.slots, f.slots)
    assert_clean_status()


def test_two_engines_on_two_streams_at_once():
    """Decode steps of two engines, one a stream, with nothing to order them."""
    engines = [Engine(rows=3, blocks=40, width=8, room=3) for _ in range(2)]
    outs = [[] for _ in engines]
    streams = [torch.cuda.Stream() for _ in engines]
    tokens = [[C.bf16(np.random.default_rng(i).standard_normal((30, 3, h, 64)), DEV) for h in (HQ, HKV, HKV)]
              for i in range(2)]
    ones = _i32([1, 1, 1])
    torch.cuda.synchronize()
    for step in range(30):
        for e, out, stream, x in zip(engines, outs, streams, tokens):
            with torch.cuda.stream(stream):
                e.new.copy_(ones)
                for t, y in zip((e.q, e.k, e.v), x):
                    t.copy_(y[step])
                e.bookkeeping()
                e.write()
                out.append(torch.zeros(3, HQ // 2, 128, dtype=torch.bfloat16, device=DEV))
                tvl.diff_attention_decode(out[-1], e.q, e.kc, e.vc, e.tables, e.lens, e.lam, 0.125)
    torch.cuda.synchronize()
    for e, out in zip(engines, outs):                     # the same again, one after the other
        f = Engine(rows=3, blocks=40, width=8, room=3)
        for step in range(30):
            f.new.copy_(ones)
            for t, y in zip((f.q, f.k, f.v), tokens[engines.index(e)]):
                t.copy_(y[step])
            f.bookkeeping()
            f.write()
            want = torch.zeros_like(out[step])
            tvl.diff_attention_decode(want, f.q, f.kc, f.vc, f.tables, f.lens, f.lam, 0.125)
            assert torch.equal(want, out[step])
        assert torch.equal(e.kc, f.kc) and torch.equal(e.tables, f.tables)
    assert_clean_status()


def test_pools_past_4_gb():
    """A step's outputs do not depend on where in the pool its blocks lie: the last blocks
    of a pool of 600000 (4.9 GB a cache, past 2^31 elements) against a small one."""
    got = []
    for blocks in (40, 600000):
        e = Engine(rows=3, blocks=40, width=12, room=160)
        if blocks > 40:
            e.kc = e.vc = e.cache = None
            e.kc, e.vc = (torch.zeros(blocks, BS, HKV, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
            e.free, e.count = torch.arange(blocks, dtype=torch.int32, device=DEV), _i32([blocks])
        outs = []
        for new in ([70, 40, 1], [20, 90, 5]):
            e.draw(new)
            e.bookkeeping()
            e.write()
            out = torch.zeros_like(e.out)
            tvl.diff_attention_prefill(out, e.q, e.qsl, e.kc, e.vc, e.tables, e.lens, e.lam, 0.125, 128, window=50,
                                       sinks=3, norm_weight=e.weight)
            outs.append(out)
        for rows in (3, 1):                               # (one launch, and with a wide table the split)
            tab = torch.full((rows, 300), -1, dtype=torch.int32, device=DEV)
            tab[:, :12] = e.tables[:rows]
            for t in (e.tables[:rows].contiguous(), tab):
                out = torch.zeros(rows, HQ // 2, 128, dtype=torch.bfloat16, device=DEV)
                tvl.diff_attention_decode(out, e.q[:rows].contiguous(), e.kc, e.vc, t, e.lens[:rows].contiguous(), e.lam,
                                          0.125, norm_weight=e.weight)
                outs.append(out)
        if blocks > 40:
            assert int(e.tables.max()) == blocks - 1
        got.append(outs)
        assert_clean_status()
    for a, b in zip(*got):
        assert torch.equal(a, b)


FIRST_CALLS = """
import torch, paged_kv_cache_198_gb300 as tvl
b = lambda *s: torch.randn(*s, device="cuda").bfloat16()
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
kc, vc, q, k = b(8, 16, 2, 64), b(8, 16, 2, 64), b(4, 8, 64), b(4, 2, 64)
tab, lens, new, free, count = i(7, 7, 7, 7).view(1, 4), i(0), i(4), torch.arange(8, dtype=torch.int32, device="cuda"), i(8)
qsl, slots, pos, axes = i(0, 0), i(0, 0, 0, 0), i(0, 0, 0, 0), torch.zeros(3, 4, dtype=torch.int32, device="cuda")
lam, po, do = torch.rand(4, device="cuda"), b(4, 4, 128), b(1, 4, 128)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    tvl.build_step_tables(tab, free, lens, qsl, slots, pos, count, lens, new, 16)
    tvl.rope_axes_paged_kv_write(q, k, k, kc, vc, slots, axes, (8, 12, 12))
    tvl.diff_attention_prefill(po, q, qsl, kc, vc, tab, lens, lam, 0.125, 4)
    tvl.diff_attention_decode(do, q[3:], kc, vc, tab, lens, lam, 0.125)
g.replay()
torch.cuda.synchronize()
assert lens.tolist() == [4] and tab[0, 0] == 7 and slots.tolist() == [112, 113, 114, 115], (lens, tab, slots)
assert (po[3].float() - do[0].float()).abs().max() < 0.05 and tvl.get_device_status() == 0
print("ok")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
