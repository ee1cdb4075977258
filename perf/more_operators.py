"""The cases on which step tables, rotary positions with several axes and
differential attention are measured.

Kinds of case (``kind``):
  tables        one engine step's bookkeeping on the GPU: rows that are done give
                their blocks back, the others get blocks for their new tokens, and
                the slot and position of every new token are written
  axes_write    rotary embedding of a batch's q and new K by positions with several
                axes (time, height, width), and the K and V rows written into the
                bf16 or the 4-bit paged cache
  diff_decode   differential attention of one token a sequence over the bf16 paged
                cache, whole context or a window with sinks
  diff_prefill  the same for chunks of new tokens, causal

Tables: the free blocks are a stack, free[0 .. count).  In the order of the rows, a
row with new < 0 pushes its blocks (in the order of its table) and ends with length
0; then the k-th new block of the step, counted over the rows and in each by
position, is the k-th from the top.  Places behind the last token hold slot -1 and
position 0.

Axes: with D = 64 there are 32 pairs (d, d + 32) at frequency theta^(-2 i / 64); the
position that turns pair i is that of its axis: the first sections[0] pairs belong
to axis 0 and so on, or, interleaved among A axes, pair i to axis i % A while
i < A * sections[i % A], and to axis 0 otherwise.

Differential attention: query heads 2 i and 2 i + 1 are the two maps of pair i, KV
heads 2 j and 2 j + 1 their two keys, with pair i reading pair j = i / group; the
value is the two V heads side by side, 128 wide.
  d = softmax(scale q1 K1) V - lambda softmax(scale q2 K2) V,
  out = out_scale * weight * d / sqrt(mean d^2 + eps)   (no weight: out_scale * d)
with lambda of the pair, or of the token and the pair.
"""
import math

import torch

own = False

D = 64
EPS = 1e-5
THETA = 500000.0
F32, F64, BF16, U8, I32 = torch.float32, torch.float64, torch.bfloat16, torch.uint8, torch.int32
REC = 1152                      # bytes of a 16-token record of the 4-bit cache
DEV = "cuda"


def listed():
    return [
        # a single conversation's next token: latency
        dict(name="tables one", kind="tables", seqs=1, lo=777, hi=777, new=1, done=0, bs=16),
        # a continuous batch of the widest kind: one token each, a few rows leave
        dict(name="tables step 256", kind="tables", seqs=256, lo=16, hi=8192, new=1, done=5, bs=32),
        # prompts of a long-context batch taken in at once
        dict(name="tables prompts 64", kind="tables", seqs=64, lo=1, hi=2000, new=8001, done=10, bs=16),
        # a decode step of a chat about images: 64 tokens into 64 scattered blocks
        dict(name="axes step 64", kind="axes_write", seqs=64, new=1, lo=500, hi=4000, hq=32, hkv=8, bs=16,
             axes="8 12 12", interleaved=False, four=False),
        # prompts with images in chunks: the bandwidth end of the write
        dict(name="axes images 16x700", kind="axes_write", seqs=16, new=700, lo=700, hi=2600, hq=32, hkv=8, bs=32,
             axes="12 10 10", interleaved=True, four=False),
        # video frames into the 4-bit cache
        dict(name="axes 4-bit 8x999", kind="axes_write", seqs=8, new=999, lo=999, hi=2600, hq=32, hkv=8, bs=16,
             axes="8 12 12", interleaved=False, four=True),
        # one short conversation on a small model: latency
        dict(name="diff one", kind="diff_decode", seqs=1, lo=777, hi=777, hq=8, hkv=2, bs=16, window=0, sinks=0,
             norm=True, per_token=False),
        # the ordinary serving batch: 64 sequences of 0.5k to 4k tokens
        dict(name="diff batch 64", kind="diff_decode", seqs=64, lo=512, hi=4096, hq=32, hkv=8, bs=16, window=0, sinks=0,
             norm=True, per_token=False),
        # long documents, lambda from the token
        dict(name="diff long 8", kind="diff_decode", seqs=8, lo=32768, hi=131072, hq=32, hkv=8, bs=16, window=0, sinks=0,
             norm=False, per_token=True),
        # a single short prompt
        dict(name="diff prefill one", kind="diff_prefill", seqs=1, new=100, lo=612, hi=612, hq=32, hkv=8, bs=16,
             window=0, sinks=0, norm=True, per_token=False),
        # chunked prefill of a mixed batch: 512 new tokens each on prefixes up to 2k
        dict(name="diff chunks 16", kind="diff_prefill", seqs=16, new=512, lo=512, hi=2560, hq=32, hkv=8, bs=16,
             window=0, sinks=0, norm=True, per_token=False),
        # long prompts, a wide window
        dict(name="diff prefill long 2", kind="diff_prefill", seqs=2, new=4096, lo=6001, hi=8192, hq=32, hkv=8, bs=32,
             window=4096, sinks=16, norm=True, per_token=True),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["tables", "axes_write", "axes_write", "diff_decode", "diff_decode", "diff_prefill",
                       "diff_prefill"])
    c = dict(kind=kind, bs=rng.choice([16, 32, 64, 128]))
    if kind == "tables":
        c["new"] = rng.choice([1, log_int(2, 10000)])
        c["seqs"] = max(1, min(1000, log_int(1, 500000) // c["new"]))
        c["lo"] = log_int(1, 300)
        c["hi"] = c["lo"] + log_int(1, 8000)
        c["done"] = rng.choice([0, 5, 30])
        return _fit(c)
    pairs = rng.choice([1, 1, 2, 3, 4, 4, 4, 6, 8])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8])
    if kind == "diff_prefill":
        pairs, group = rng.choice([1, 2, 4, 4, 8]), rng.choice([1, 2, 4, 4, 8])
    while pairs * group > 32:
        group = max(1, group // 2)
    c.update(hq=2 * pairs * group, hkv=2 * pairs)
    if kind == "axes_write":
        c["new"] = rng.choice([1, log_int(2, 900)])
        c["seqs"] = max(1, min(256, log_int(1, 90000 // c["hkv"]) // c["new"]))
        c["lo"] = c["new"] + rng.randrange(0, 300)
        c["hi"] = c["lo"] + log_int(1, 2000)
        c["axes"], c["interleaved"] = rng.choice([("8 12 12", False), ("12 10 10", True), ("16 16", False),
                                                  ("11 11 10", True), ("32", False), ("2 10 10 10", False)])
        c["four"] = rng.random() < 0.4
        return _fit(c)
    c["window"] = log_int(16, 16384) if rng.random() < 0.4 else 0
    c["sinks"] = rng.choice([0, 1, 4, 16, log_int(1, 100)]) if c["window"] else 0
    c["norm"], c["per_token"] = rng.random() < 0.7, rng.random() < 0.4
    if kind == "diff_prefill":
        c["new"] = log_int(1, 3000)
        c["seqs"] = max(1, min(32, int(rng.uniform(0.1, 1.0) * 60000) // (c["new"] + 1500)))
        c["lo"] = c["new"]
        c["hi"] = c["new"] + log_int(1, 3000)
        return _fit(c)
    c["hi"] = log_int(1, 100000)
    seen = min(c["hi"], c["window"] + c["sinks"]) if c["window"] else c["hi"]
    c["seqs"] = max(1, min(300, log_int(100, 500000) * 8 // c["hkv"] // seen))
    c["lo"] = max(1, int(c["hi"] * rng.uniform(0.02, 1.0)))
    return _fit(c)


def _cost(c):
    """What a case must not have more of than the largest listed one of its kind:
    bytes, operations, cached rows, scores of the plain form, table entries."""
    w = work(c)
    rows = sum(_lens(c)) * c["hkv"] if "hkv" in c else 0
    scores = c["seqs"] * c["hq"] * c["new"] * c["hi"] if c["kind"] == "diff_prefill" else 0
    entries = c["seqs"] * (c["hi"] + c["new"]) // c["bs"] if c["kind"] == "tables" else 0
    return w["bytes"], w["flops"], rows, scores, entries


def _fit(c):
    most = [max(x) for x in zip(*(_cost(k) for k in listed() if k["kind"] == c["kind"]))]
    while any(x > y for x, y in zip(_cost(c), most)):
        if c["seqs"] > 1:
            c["seqs"] = c["seqs"] * 3 // 4
        else:
            c["hi"] = max(c["hi"] * 3 // 4, c.get("new", 1))
            if "new" in c:
                c["new"] = max(1, c["new"] * 3 // 4)
            c["lo"] = min(c["lo"], c["hi"])
    return c


# ------------------------------------------------------------------- inputs


def _lens(c):
    """The case's context lengths, spread over [lo, hi] (over the logarithm
    where that spans more than a factor of ten)."""
    lo, hi, out = c["lo"], c["hi"], []
    for i in range(c["seqs"]):
        f = (0.31 + 0.6180339887498949 * i) % 1.0
        x = lo * (hi / lo) ** f if hi > 10 * lo else lo + (hi - lo) * f
        out.append(max(1, int(round(x))))
    return out


def _new_tokens(c):
    """Tables: new tokens of each row; -1: the row is done."""
    out = []
    for i in range(c["seqs"]):
        n = c["new"] if c["new"] == 1 else max(1, round(c["new"] * (0.25 + 0.75 * ((0.77 + 0.7548776662 * i) % 1.0))))
        out.append(-1 if c["done"] and (i * 37 + 11) % 100 < c["done"] else n)
    return out


def _visible(c, n):
    """Tokens that the last of n positions sees."""
    w, s = c["window"], c["sinks"]
    return n if w == 0 or n <= w else w + min(s, n - w)


def _axis_of(c):
    """Axis of each of the 32 pairs."""
    sec = [int(x) for x in c["axes"].split()]
    a = len(sec)
    if c["interleaved"]:
        return [i % a if i < a * sec[i % a] else 0 for i in range(D // 2)]
    return [j for j in range(a) for _ in range(sec[j])]


def _randn(gen, *shape):
    """Normal values without the far tail, as after a norm."""
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).clamp_(-2.2, 2.2).to(BF16)


def _pool(gen, nb, bs, hkv):
    """A 4-bit cache with a used block's contents everywhere."""
    pool = torch.empty(nb, bs // 16, hkv, REC, dtype=U8, device=DEV)
    pool[..., :1024] = torch.randint(0, 256, (nb, bs // 16, hkv, 1024), generator=gen, device=DEV, dtype=U8)
    s = torch.rand(nb, bs // 16, hkv, 32, 1, generator=gen, device=DEV).mul_(0.12).add_(0.24)
    z = s * (torch.rand(s.shape, generator=gen, device=DEV).mul_(1.5).sub_(8.2))
    pool[..., 1024:] = torch.cat([s, z], dim=-1).to(BF16).view(U8).reshape(nb, bs // 16, hkv, 128)
    return pool


def _deal(gen, lens, bs, width):
    """Scattered blocks: tables [n, width], the permutation of all blocks, how many are used."""
    blocks = [-(-x // bs) for x in lens]
    used = sum(blocks)
    nb = used + used // 4 + 1
    perm = torch.randperm(nb, generator=gen, device=DEV).to(I32)
    tables = torch.full((len(lens), width), -1, dtype=I32, device=DEV)
    at = torch.arange(width, device=DEV)[None] < torch.tensor(blocks, device=DEV)[:, None]
    tables[at] = perm[:used]
    return tables, perm, used


def _prepare_tables(c, gen):
    bs, lens, new = c["bs"], _lens(c), _new_tokens(c)
    total = sum(max(0, x) for x in new)
    blocks = [-(-x // bs) for x in lens]
    need = sum(-(-(x + y) // bs) - b for x, y, b in zip(lens, new, blocks) if y > 0)
    width = max(-(-(x + max(0, y)) // bs) for x, y in zip(lens, new)) + 3
    used = sum(blocks)
    nb = used + need + need // 3 + 5
    perm = torch.randperm(nb, generator=gen, device=DEV).to(I32)
    tables = torch.full((len(lens), width), -1, dtype=I32, device=DEV)
    at = torch.arange(width, device=DEV)[None] < torch.tensor(blocks, device=DEV)[:, None]
    tables[at] = perm[:used]
    free = torch.full((nb,), -1, dtype=I32, device=DEV)
    free[:nb - used] = perm[used:]
    room = -(-total // 64) * 64                       # a captured step's padded token count
    st = dict(case=dict(c), tables=tables, free=free, room=room,
              count=torch.tensor([nb - used], dtype=I32, device=DEV), lens=torch.tensor(lens, dtype=I32, device=DEV),
              new=torch.tensor(new, dtype=I32, device=DEV))
    st["out"] = dict(context_lens=torch.zeros(len(lens), dtype=I32, device=DEV),
                     query_start_loc=torch.zeros(len(lens) + 1, dtype=I32, device=DEV),
                     slot_mapping=torch.zeros(room, dtype=I32, device=DEV),
                     positions=torch.zeros(room, dtype=I32, device=DEV),
                     free_count=torch.zeros(1, dtype=I32, device=DEV))
    return st


def _axes_positions(c, pos, gen):
    """[axes, T]: a third of a chunk is text (all axes alike), the rest rows of 28
    patches; pos [n, new] are the tokens' places in their sequences."""
    a = len(c["axes"].split())
    out = pos[None].repeat(a, 1, 1)
    text = c["new"] // 3 + 1
    if c["new"] > text and a > 1:
        patch = torch.arange(c["new"] - text, device=DEV)
        first = pos[:, text:text + 1]
        out[0, :, text:] = first + (patch // 784 if a > 2 else patch // 28)
        out[1, :, text:] = first + (patch % 784 // 28 if a > 2 else patch % 28)
        if a > 2:
            out[2, :, text:] = first + patch % 28
    return out.reshape(a, -1).to(I32).contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if c["kind"] == "tables":
        st = _prepare_tables(c, gen)
        if own:
            st["call"] = _bind(st)
        return st
    bs, hq, hkv, lens = c["bs"], c["hq"], c["hkv"], _lens(c)
    n = c["seqs"]
    mb = max(-(-x // bs) for x in lens)
    tables, perm, used = _deal(gen, lens, bs, mb)
    nb = perm.numel()
    ctx = torch.tensor(lens, dtype=I32, device=DEV)
    st = dict(case=dict(c), tables=tables, ctx=ctx, scale=1.0 / math.sqrt(D))
    if c["kind"] == "axes_write":
        new = c["new"]
        pos = (ctx[:, None] - new + torch.arange(new, device=DEV)).clamp_(min=0)
        page = torch.gather(tables, 1, pos // bs)
        st["positions"] = _axes_positions(c, pos, gen)
        st["slots"] = (page * bs + pos % bs).reshape(-1).to(I32)
        t = n * new
        st["q"], st["k"], st["v"] = _randn(gen, t, hq, D), _randn(gen, t, hkv, D), _randn(gen, t, hkv, D)
        if c["four"]:
            st["pool"] = _pool(gen, nb, bs, hkv)
            st["src"] = torch.unique(page).to(I32)
            st["dst"] = torch.arange(st["src"].numel(), dtype=I32, device=DEV)
            st["k_out"] = torch.zeros(st["src"].numel(), bs, hkv, D, dtype=BF16, device=DEV)
            st["v_out"] = torch.zeros_like(st["k_out"])
        else:
            st["k_out"], st["v_out"] = _randn(gen, nb, bs, hkv, D), _randn(gen, nb, bs, hkv, D)
    else:
        rows = n * c["new"] if c["kind"] == "diff_prefill" else n
        pairs = hq // 2
        st["q"] = (_randn(gen, rows, hq, D) * 1.5).to(BF16)
        st["k"], st["v"] = _randn(gen, nb, bs, hkv, D), _randn(gen, nb, bs, hkv, D)
        shape = (rows, pairs) if c["per_token"] else (pairs,)
        st["lam"] = torch.rand(shape, generator=gen, device=DEV).mul_(0.6).add_(0.2)
        st["weight"] = torch.rand(2 * D, generator=gen, device=DEV).add_(0.5).to(BF16) if c["norm"] else None
        st["out_scale"] = 0.4 if c["norm"] else 1.0
        if c["kind"] == "diff_prefill":
            st["starts"] = torch.arange(n + 1, dtype=I32, device=DEV) * c["new"]
        st["out"] = torch.zeros(rows, pairs, 2 * D, dtype=BF16, device=DEV)
    if own:
        st["call"] = _bind(st)
    return st


# ------------------------------------------------------- the framework's calls


def _bind(st):
    import paged_kv_cache_198_gb300 as tvl

    c = st["case"]
    if c["kind"] == "tables":
        o = st["out"]
        return [tvl.bind_build_step_tables(st["tables"], st["free"], o["context_lens"], o["query_start_loc"],
                                           o["slot_mapping"], o["positions"], st["count"], st["lens"], st["new"],
                                           c["bs"], free_count_out=o["free_count"])]
    if c["kind"] == "axes_write":
        sections = [int(x) for x in c["axes"].split()]
        if c["four"]:
            return [tvl.bind_kv4_axes_write(st["k"], st["v"], st["pool"], st["slots"], st["q"], st["positions"],
                                            sections, interleaved=c["interleaved"], rope_theta=THETA),
                    tvl.bind_kv4_expand_blocks(st["k_out"], st["v_out"], st["pool"], st["src"], st["dst"])]
        return [tvl.bind_rope_axes_paged_kv_write(st["q"], st["k"], st["v"], st["k_out"], st["v_out"], st["slots"],
                                                  st["positions"], sections, interleaved=c["interleaved"],
                                                  rope_theta=THETA)]
    more = dict(window=c["window"], sinks=c["sinks"], norm_weight=st["weight"], norm_eps=EPS,
                out_scale=st["out_scale"])
    if c["kind"] == "diff_decode":
        return [tvl.bind_diff_attention_decode(st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"], st["lam"],
                                               st["scale"], **more)]
    return [tvl.bind_diff_attention_prefill(st["out"], st["q"], st["starts"], st["k"], st["v"], st["tables"],
                                            st["ctx"], st["lam"], st["scale"], c["new"], **more)]


def _outputs(st):
    kind = st["case"]["kind"]
    if kind == "tables":
        return dict(st["out"], block_tables=st["tables"], free_blocks=st["free"])
    if kind == "axes_write":
        return {"q": st["q"], "k": st["k_out"], "v": st["v_out"]}
    return st["out"]


def run(state):
    if own:
        for call in state["call"]:
            call()
        return _outputs(state)
    kind = state["case"]["kind"]
    if kind == "tables":
        return _plain_tables(state)
    if kind == "axes_write":
        return _plain_write(state)
    if kind == "diff_decode":
        return _plain_decode(state)
    return _plain_prefill(state)


# ------------------------------------------------------------ the plain forms


def _plain_tables(st):
    bs, tables, free = st["case"]["bs"], st["tables"].long(), st["free"].long()
    lens, new, count = st["lens"].long(), st["new"].long(), st["count"].long()
    rows, width = tables.shape
    col = torch.arange(width, device=DEV)[None]
    had = (lens + bs - 1) // bs
    done = new < 0
    # blocks of the rows that are done, onto the stack; the last place takes the rest
    give = done[:, None] & (col < had[:, None])
    place = torch.where(give, count + torch.cumsum(give.reshape(-1), 0).reshape(rows, width) - 1, free.numel())
    free = torch.cat([free, free[:1]])
    free[place] = tables
    free = free[:-1]
    top = count + give.sum()
    add = new.clamp(min=0)
    ctx = torch.where(done, 0, lens + add)
    need = torch.where(done, 0, (ctx + bs - 1) // bs - had)
    nth = (torch.cumsum(need, 0) - need)[:, None] + col - had[:, None]
    fresh = ~done[:, None] & (col >= had[:, None]) & (col < (had + need)[:, None])
    tables = torch.where(fresh, free[torch.where(fresh, top - 1 - nth, 0)], tables)
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(add, 0)])
    i = torch.arange(st["room"], device=DEV)
    s = torch.searchsorted(start[1:], i, right=True)
    live = s < rows
    s = s.clamp(max=rows - 1)
    pos = torch.where(live, ctx[s] - start[s + 1] + i, 0)
    slot = torch.where(live, tables[s, pos // bs] * bs + pos % bs, -1)
    return dict(context_lens=ctx.to(I32), query_start_loc=start.to(I32), slot_mapping=slot.to(I32),
                positions=pos.to(I32), free_count=(top - need.sum()).to(I32), block_tables=tables.to(I32),
                free_blocks=free.to(I32))


def _plain_rope(x, pos, axis):
    """Angles in 64 bits (positions are far), the rotation in 32."""
    inv = THETA ** (-torch.arange(D // 2, dtype=F64, device=DEV) * 2.0 / D)
    a = (pos.to(F64)[axis].T * inv)[:, None]
    cos, sin = torch.cos(a).to(F32), torch.sin(a).to(F32)
    x0, x1 = x[..., :D // 2].to(F32), x[..., D // 2:].to(F32)
    return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], dim=-1).to(BF16)


def _plain_quantise(x):
    """Codes [T, Hkv, 32] in bytes and (s, z) [T, Hkv, 2] in bf16 of rows [T, Hkv, 64]."""
    x = x.to(F32)
    z = x.amin(dim=-1, keepdim=True)
    s = (x.amax(dim=-1, keepdim=True) - z) / torch.full_like(z, 15.0)   # a quotient, not a product with 1 / 15
    s = ((s.view(I32) + 0xFFFF) & -0x10000).view(F32)                   # up to the next bf16
    code = torch.round(torch.where(s > 0, (x - z) / s, 0.0)).clamp_(0, 15).to(U8)
    return code[..., 0::2] + code[..., 1::2] * 16, torch.cat([s, z], dim=-1).to(BF16)


def _plain_values(pool):
    """The values [NB, bs, Hkv, 64] x 2 that a 4-bit cache stands for, in 32 bits."""
    nb, chunks, hkv = pool.shape[:3]
    out = []
    for part in (0, 1):
        code = pool[..., 512 * part:512 * part + 512].reshape(nb, chunks, hkv, 16, 32)
        meta = pool[..., 1024 + 64 * part:1088 + 64 * part].contiguous().view(BF16).to(F32).reshape(nb, chunks, hkv, 16, 2)
        x = torch.stack([code & 15, code >> 4], dim=-1).reshape(nb, chunks, hkv, 16, D).to(F32)
        x = x.mul_(meta[..., :1]).add_(meta[..., 1:])
        out.append(x.transpose(2, 3).reshape(nb, chunks * 16, hkv, D))
    return out


def _plain_write(st):
    c, slots = st["case"], st["slots"].long()
    bs = c["bs"]
    axis = torch.tensor(_axis_of(c), device=DEV)
    st["q"].copy_(_plain_rope(st["q"], st["positions"], axis))
    k, v = _plain_rope(st["k"], st["positions"], axis), st["v"]
    if not c["four"]:
        st["k_out"].view(-1, c["hkv"], D)[slots] = k
        st["v_out"].view(-1, c["hkv"], D)[slots] = v
        return _outputs(st)
    pool = st["pool"]
    page, sub, tok = slots // bs, slots % bs // 16, slots % 16
    for part, x in ((0, k), (1, v)):
        code, meta = _plain_quantise(x)
        pool[..., 512 * part:512 * part + 512].unflatten(-1, (16, 32))[page, sub, :, tok] = code
        pool[..., 1024 + 64 * part:1088 + 64 * part].unflatten(-1, (16, 4))[page, sub, :, tok] = meta.view(U8)
    k, v = _plain_values(pool[st["src"].long()])
    return {"q": st["q"], "k": k.to(BF16), "v": v.to(BF16)}


def _plain_difference(st, o):
    """o [rows, pairs, 2, 128] in 32 bits: the two maps' outputs."""
    lam = st["lam"].expand(o.shape[:2])[..., None]
    d = o[:, :, 0] - lam * o[:, :, 1]
    if st["weight"] is not None:
        d = d / torch.sqrt(torch.mean(d * d, dim=-1, keepdim=True) + EPS) * st["weight"].to(F32)
    return (d * st["out_scale"]).to(BF16)


def _plain_decode(st):
    c, ctx = st["case"], st["ctx"].long()
    n, kvp, bs, w, sinks = len(ctx), c["hkv"] // 2, c["bs"], c["window"], c["sinks"]
    most = max(_visible(c, x) for x in _lens(c))
    j = torch.arange(most, device=DEV)[None]
    first = (ctx - w).clamp(min=0)[:, None] if w else torch.zeros_like(ctx)[:, None]
    kept = first.clamp(max=sinks)                             # sinks ahead of the window
    pos = torch.where(j < kept, j, j - kept + first)
    seen = pos < ctx[:, None]
    pos = torch.where(seen, pos, 0)
    slot = torch.gather(st["tables"].long(), 1, pos // bs) * bs + pos % bs
    k = st["k"].view(-1, kvp, 2, D)[slot].to(F32)
    v = st["v"].view(-1, kvp, 2 * D)[slot].to(F32)
    q = st["q"].to(F32).reshape(n, kvp, -1, 2, D)
    s = (torch.einsum("shgmd,snhmd->shgmn", q, k) * st["scale"]).masked_fill_(~seen[:, None, None, None], -math.inf)
    p = torch.exp(s - s.amax(dim=-1, keepdim=True))
    o = torch.einsum("shgmn,snhe->shgme", p, v) / p.sum(dim=-1, keepdim=True)
    return _plain_difference(st, o.reshape(n, c["hq"] // 2, 2, 2 * D))


def _plain_prefill(st):
    c, ctx = st["case"], st["ctx"].long()
    n, kvp, bs, new, w = len(ctx), c["hkv"] // 2, c["bs"], c["new"], c["window"]
    key = torch.arange(int(st["tables"].shape[1]) * bs, device=DEV)
    page = st["tables"].long().clamp(min=0)
    k = st["k"][page].reshape(n, -1, kvp, 2, D).to(F32)
    v = st["v"][page].reshape(n, -1, kvp, 2 * D).to(F32)
    q = st["q"].to(F32).reshape(n, new, kvp, -1, 2, D)
    at = (ctx[:, None] - new + torch.arange(new, device=DEV))[:, :, None]
    seen = key <= at
    if w:
        seen &= (key > at - w) | (key < c["sinks"])
    s = torch.einsum("sthgmd,snhmd->shgmtn", q, k).mul_(st["scale"])
    s.masked_fill_(~seen[:, None, None, None], -math.inf)
    p = s.sub_(s.amax(dim=-1, keepdim=True)).exp_()
    o = torch.einsum("shgmtn,snhe->sthgme", p.div_(p.sum(dim=-1, keepdim=True)), v)
    return _plain_difference(st, o.reshape(n * new, c["hq"] // 2, 2, 2 * D))


# ---------------------------------------------------------------------- work


def work(case):
    c, lens, n = case, _lens(case), case["seqs"]
    if c["kind"] == "tables":
        new = _new_tokens(c)
        total = sum(max(0, x) for x in new)
        had = [-(-x // c["bs"]) for x in lens]
        given = sum(b for b, y in zip(had, new) if y < 0)
        taken = sum(-(-(x + y) // c["bs"]) - b for x, y, b in zip(lens, new, had) if y >= 0)
        # a slot and a position a token; lengths in, lengths and starts out; blocks moved
        return {"bytes": 8 * (-(-total // 64) * 64) + 16 * n + 8 * (given + taken) + 12, "flops": 0}
    hq, hkv = c["hq"], c["hkv"]
    if c["kind"] == "axes_write":
        t, new, bs = n * c["new"], c["new"], c["bs"]
        meta = 4 * t * (len(c["axes"].split()) + 1)
        if not c["four"]:
            return {"bytes": t * (2 * hq * 128 + 4 * hkv * 128) + meta, "flops": 0}
        # each new row read, each code written; the touched blocks read and expanded
        blocks = sum((x - 1) // bs - max(0, x - new) // bs + 1 for x in lens)
        return {"bytes": t * (2 * hkv * 128 + 2 * hq * 128 + hkv * 72) + blocks * bs * hkv * (72 + 256) + meta, "flops": 0}
    if c["kind"] == "diff_prefill":
        pairs = sum(_visible(c, p + 1) for x in lens for p in range(x - c["new"], x))
        keys = sum(min(x, c["window"] + c["new"] - 1 + c["sinks"]) if c["window"] else x for x in lens)
        lam = 2 * hq * (n * c["new"] if c["per_token"] else 1)
        # a score of 64 products and 128 of the value, for every query head
        return {"bytes": keys * hkv * 256 + n * c["new"] * hq * 256 + lam, "flops": 6 * D * hq * pairs}
    seen = sum(_visible(c, x) for x in lens)
    return {"bytes": seen * hkv * 256 + n * hq * D * 4 + 4 * n + 4 * (seen // c["bs"]), "flops": 6 * D * hq * seen}


# -------------------------------------------------------------- in 64 bits


def _exact_tables(st):
    """Row by row on the host, from the definition."""
    bs = st["case"]["bs"]
    tables, free = st["tables"].cpu().numpy().copy(), st["free"].cpu().numpy().copy()
    lens, new, top = st["lens"].tolist(), st["new"].tolist(), int(st["count"])
    for s, n in enumerate(new):
        if n < 0:
            b = -(-lens[s] // bs)
            free[top:top + b] = tables[s, :b]
            top += b
            lens[s] = 0
    start, slots, positions = [0], [], []
    for s, n in enumerate(new):
        n = max(0, n)
        had, all_ = -(-lens[s] // bs), -(-(lens[s] + n) // bs)
        if new[s] >= 0:
            tables[s, had:all_] = free[top - (all_ - had):top][::-1]
            top -= all_ - had
        pos = torch.arange(lens[s], lens[s] + n)
        positions.append(pos)
        slots.append(torch.from_numpy(tables[s].astype("int64"))[pos // bs] * bs + pos % bs)
        lens[s] += n
        start.append(start[-1] + n)
    pad = torch.zeros(st["room"] - start[-1], dtype=torch.int64)
    out = dict(context_lens=torch.tensor(lens), query_start_loc=torch.tensor(start),
               slot_mapping=torch.cat(slots + [pad - 1]), positions=torch.cat(positions + [pad]),
               free_count=torch.tensor([top]), block_tables=torch.from_numpy(tables), free_blocks=torch.from_numpy(free))
    return {k: v.to(I32).to(DEV) for k, v in out.items()}


def _exact_write(st):
    c = st["case"]
    sec = [int(x) for x in c["axes"].split()]
    freq = torch.exp(-torch.arange(32, dtype=F64, device=DEV) / 32.0 * math.log(THETA))
    angle = torch.zeros(st["positions"].shape[1], 32, dtype=F64, device=DEV)
    end = 0
    for a, n in enumerate(sec):
        if c["interleaved"]:
            # every A-th pair from a on, n of them; axis 0 has what is left
            mine = [i for i in range(32) if i % len(sec) == a][:n] if a else \
                [i for i in range(32) if all(i not in range(b, len(sec) * m, len(sec)) for b, m in enumerate(sec) if b)]
        else:
            mine = list(range(end, end + n))
            end += n
        angle[:, mine] = st["positions"][a].to(F64)[:, None] * freq[mine]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotate(x):
        z = torch.view_as_complex(torch.stack([x[..., :32], x[..., 32:]], dim=-1).to(F64)) * turn
        return torch.cat([z.real, z.imag], dim=-1)

    got, slot = {"q": rotate(st["q"])}, st["slots"].long()
    bs, hkv = c["bs"], c["hkv"]
    if not c["four"]:
        for name, x in (("k", rotate(st["k"])), ("v", st["v"].to(F64))):
            new = st[name + "_out"].to(F64).reshape(-1, hkv, D)
            new[slot] = x
            got[name] = new.reshape(-1, bs, hkv, D)
        return got
    src = st["src"].long()
    place = torch.zeros(int(st["pool"].shape[0]), dtype=torch.int64, device=DEV)
    place[src] = torch.arange(src.numel(), device=DEV)
    to = place[slot // bs] * bs + slot % bs
    rec = st["pool"][src]                              # [blocks, bs / 16, Hkv, 1152]
    d = torch.arange(D, device=DEV)
    # the rotated K is a bf16 row before it is quantised
    for name, part, x in (("k", 0, rotate(st["k"]).to(BF16).to(F64)), ("v", 1, st["v"].to(F64))):
        rows = []
        for tok in range(16):
            code = rec[..., 512 * part + 32 * tok:512 * part + 32 * tok + 32][..., d // 2].to(torch.int64) >> (4 * (d % 2)) & 15
            sz = rec[..., 1024 + 64 * part + 4 * tok:1028 + 64 * part + 4 * tok].contiguous().view(BF16).to(F64)
            rows.append(sz[..., :1] * code.to(F64) + sz[..., 1:])
        old = torch.stack(rows, dim=2).reshape(-1, hkv, D)
        z, top = x.min(dim=-1, keepdim=True).values, x.max(dim=-1, keepdim=True).values
        m, e = torch.frexp((top - z) / torch.full_like(z, 15.0))
        two_e = ((e.to(torch.int64) + 1015) << 52).view(F64)  # 2 ** (e - 8), exactly
        s = torch.ceil(m * 256.0) * two_e                     # 8 significant bits, upwards
        code = torch.where(s > 0, torch.round((x - z) / s), 0.0).clamp(0, 15)
        old[to] = s * code + z
        got[name] = old.reshape(-1, bs, hkv, D)
    return got


def _exact_attention(st):
    c = st["case"]
    bs, new, w, pairs = c["bs"], c.get("new", 1), c["window"], c["hq"] // 2
    group = pairs // (c["hkv"] // 2)
    out = torch.zeros(c["seqs"] * new, pairs, 2 * D, dtype=F64, device=DEV)
    lam = st["lam"].to(F64).expand(c["seqs"] * new, pairs)
    for s, n in enumerate(_lens(c)):
        first = max(0, n - new - w + 1) if w else 0
        keep = min(c["sinks"], first) if w else 0
        pos = torch.cat([torch.arange(0, keep, device=DEV), torch.arange(first, n, device=DEV)])
        page, off = st["tables"][s].long()[pos // bs], pos % bs
        for i in range(pairs):
            j = i // group
            v = torch.cat([st["v"][page, off, 2 * j], st["v"][page, off, 2 * j + 1]], dim=-1).to(F64)
            k = [st["k"][page, off, 2 * j + m].to(F64) for m in (0, 1)]
            for r0 in range(s * new, s * new + new, 2048):
                r1 = min(s * new + new, r0 + 2048)
                at = torch.arange(n - new + r0 - s * new, n - new + r1 - s * new, device=DEV)[:, None]
                ok = pos <= at
                if w:
                    ok = ok & ((at - pos < w) | (pos < c["sinks"]))
                o = [torch.softmax((st["q"][r0:r1, 2 * i + m].to(F64) @ k[m].T * st["scale"]).masked_fill(~ok, -math.inf),
                                   dim=-1) @ v for m in (0, 1)]
                out[r0:r1, i] = o[0] - lam[r0:r1, i, None] * o[1]
    if st["weight"] is not None:
        out *= torch.rsqrt(out.square().mean(dim=-1, keepdim=True) + EPS) * st["weight"].to(F64)
    return out * st["out_scale"]


def exact(case, seed):
    st = prepare({k: v for k, v in case.items() if k != "name"}, seed)
    if case["kind"] == "tables":
        return _exact_tables(st)
    return _exact_write(st) if case["kind"] == "axes_write" else _exact_attention(st)
