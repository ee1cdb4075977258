"""The cases on which the 4-bit cache and the windowed attention are measured.

Kinds of case (``kind``):
  kv4_write      RoPE of a batch's q and new K, the new K and V rows quantised to
                 4 bits into their cache slots, and the touched blocks expanded
                 back to bf16 (what a prefill over a 4-bit prefix reads)
  kv4_decode     decode attention over the 4-bit paged cache, whole context or
                 a window with sinks
  window_decode  decode attention over the bf16 paged cache, window and sinks
  window_prefill chunked causal prefill over the bf16 paged cache, window and
                 sinks, bf16 output

A 4-bit cache block holds, per 16 tokens and KV head, one 1152-byte record:
K codes [16][32], V codes [16][32] (two 4-bit codes a byte, the even dimension
in the low half), K (s, z) [16][2] and V (s, z) [16][2] in bf16; a code c
stands for s * c + z.
"""
import math

import torch

own = False

D = 64
REC = 1152                      # bytes of a 16-token record
F32, F64, BF16, U8 = torch.float32, torch.float64, torch.bfloat16, torch.uint8
DEV = "cuda"


def listed():
    return [
        # one decode step of a 64-sequence batch: 64 tokens into 64 scattered blocks
        dict(name="write step 64", kind="kv4_write", seqs=64, new=1, lo=500, hi=4000, hq=32, hkv=8, bs=16),
        # prefill chunks of ragged prompts, 8 KV heads: the bandwidth end of the write
        dict(name="write chunks 16x700", kind="kv4_write", seqs=16, new=700, lo=700, hi=2600, hq=32, hkv=8, bs=32),
        # one short conversation on a small model: latency
        dict(name="kv4 one", kind="kv4_decode", seqs=1, lo=777, hi=777, hq=8, hkv=2, bs=16, window=0, sinks=0),
        # the ordinary serving batch: 64 sequences of 0.5k to 4k tokens
        dict(name="kv4 batch 64", kind="kv4_decode", seqs=64, lo=512, hi=4096, hq=32, hkv=8, bs=16, window=0, sinks=0),
        # long documents, where the 4-bit cache pays most
        dict(name="kv4 long 8", kind="kv4_decode", seqs=8, lo=32768, hi=131072, hq=32, hkv=8, bs=16, window=0, sinks=0),
        # streaming chats of very different age: window and sinks over 4 bits, groups of 8
        dict(name="kv4 window 256", kind="kv4_decode", seqs=256, lo=16, hi=8192, hq=64, hkv=8, bs=32, window=2048, sinks=4),
        # one chat inside its window: latency
        dict(name="window one", kind="window_decode", seqs=1, lo=5000, hi=5000, hq=32, hkv=8, bs=16, window=512, sinks=4),
        # a continuous batch with windowed layers
        dict(name="window batch 256", kind="window_decode", seqs=256, lo=16, hi=8192, hq=32, hkv=8, bs=32, window=1024, sinks=4),
        # long streams, a wide window, every query head with its own KV head
        dict(name="window long 8", kind="window_decode", seqs=8, lo=32768, hi=131072, hq=16, hkv=16, bs=64, window=16384, sinks=64),
        # a single short prompt
        dict(name="prefill one", kind="window_prefill", seqs=1, new=100, lo=612, hi=612, hq=32, hkv=8, bs=16, window=256, sinks=4),
        # chunked prefill of a mixed batch: 512 new tokens each on prefixes up to 2k
        dict(name="prefill chunks 16", kind="window_prefill", seqs=16, new=512, lo=512, hi=2560, hq=32, hkv=8, bs=16, window=1024, sinks=4),
        # long prompts, a wide window
        dict(name="prefill long 2", kind="window_prefill", seqs=2, new=4096, lo=6001, hi=8192, hq=32, hkv=8, bs=32, window=2048, sinks=16),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["kv4_write", "kv4_decode", "kv4_decode", "window_decode", "window_decode",
                       "window_prefill", "window_prefill"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 8, 12, 16])
    group = rng.choice([1, 2, 3, 4, 4, 6, 8])
    bs = rng.choice([16, 32, 64, 128])
    if kind == "window_prefill":
        hkv, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 4, 4, 8])
    while hkv * group > 64:
        group = max(1, group // 2)
    c = dict(kind=kind, hq=hkv * group, hkv=hkv, bs=bs)
    if kind == "kv4_write":
        c["new"] = rng.choice([1, log_int(2, 900)])
        c["seqs"] = max(1, min(256, log_int(1, 90000 // hkv) // c["new"]))
        c["lo"] = c["new"] + rng.randrange(0, 300)
        c["hi"] = c["lo"] + log_int(1, 2000)
        return _fit(c)
    c["window"] = log_int(16, 16384) if kind != "kv4_decode" or rng.random() < 0.5 else 0
    c["sinks"] = rng.choice([0, 1, 4, 16, log_int(1, 100)]) if c["window"] else 0
    if kind == "window_prefill":
        c["new"] = log_int(1, 3000)
        c["seqs"] = max(1, min(32, int(rng.uniform(0.1, 1.0) * 60000) // (c["new"] + 1500)))
        c["lo"] = c["new"]
        c["hi"] = c["new"] + log_int(1, 3000)
        return _fit(c)
    c["hi"] = log_int(1, 100000)
    seen = min(c["hi"], c["window"] + c["sinks"]) if c["window"] else c["hi"]
    c["seqs"] = max(1, min(300, log_int(100, 500000) * 8 // hkv // seen))
    c["lo"] = max(1, int(c["hi"] * rng.uniform(0.02, 1.0)))
    return _fit(c)


def _cost(c):
    """(bytes, operations, cached rows, scores of the plain form): what a case
    must not have more of than the largest listed one of its kind."""
    w = work(c)
    scores = c["seqs"] * c["hq"] * c["new"] * c["hi"] if c["kind"] == "window_prefill" else 0
    return w["bytes"], w["flops"], sum(_lens(c)) * c["hkv"], scores


def _fit(c):
    most = [max(x) for x in zip(*(_cost(k) for k in listed() if k["kind"] == c["kind"]))]
    while any(x > y for x, y in zip(_cost(c), most)):
        if c["seqs"] > 1:
            c["seqs"] = c["seqs"] * 3 // 4
        else:
            c["hi"] = max(c["hi"] * 3 // 4, c.get("new", 1))
            c["new"] = max(1, c["new"] * 3 // 4) if "new" in c else None
            c["lo"] = min(c["lo"], c["hi"])
            c = {k: v for k, v in c.items() if v is not None}
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


def _visible(c, n):
    """Tokens that the last of n positions sees."""
    w, s = c["window"], c["sinks"]
    return n if w == 0 or n <= w else w + min(s, n - w)


def _codes(gen, shape):
    """Bytes of two 4-bit codes, each spread like a quantised normal variable."""
    def half():
        return torch.randn(shape, generator=gen, device=DEV, dtype=BF16).mul_(3.2).add_(7.5).round_().clamp_(0, 15).to(U8)
    return half().add_(half().mul_(16))


def _pool(gen, nb, bs, hkv):
    """A 4-bit cache with a used block's contents everywhere."""
    pool = torch.empty(nb, bs // 16, hkv, REC, dtype=U8, device=DEV)
    pool[..., :1024] = _codes(gen, (nb, bs // 16, hkv, 1024))
    s = torch.rand(nb, bs // 16, hkv, 32, 1, generator=gen, device=DEV).mul_(0.12).add_(0.24)
    z = s * (torch.rand(s.shape, generator=gen, device=DEV).mul_(1.5).sub_(8.2))
    pool[..., 1024:] = torch.cat([s, z], dim=-1).to(BF16).view(U8).reshape(nb, bs // 16, hkv, 128)
    return pool


def _randn(gen, *shape):
    """Normal values without the far tail, as after a norm."""
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32).clamp_(-2.2, 2.2).to(BF16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    bs, hq, hkv, lens = c["bs"], c["hq"], c["hkv"], _lens(c)
    n = c["seqs"]
    blocks = [-(-x // bs) for x in lens]
    mb, used = max(blocks), sum(blocks)
    nb = used + used // 4 + 1
    perm = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    tables = torch.full((n, mb), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(mb, device=DEV)[None] < torch.tensor(blocks, device=DEV)[:, None]
    tables[at] = perm[:used]
    ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st = dict(case=dict(c), tables=tables, ctx=ctx, scale=1.0 / math.sqrt(D))
    if c["kind"] == "kv4_write":
        new = c["new"]
        pos = (ctx[:, None] - new + torch.arange(new, device=DEV)).clamp_(min=0)
        page = torch.gather(tables, 1, pos // bs)
        st["positions"] = pos.reshape(-1).to(torch.int32)
        st["slots"] = (page * bs + pos % bs).reshape(-1).to(torch.int32)
        t = n * new
        st["q"], st["k"], st["v"] = _randn(gen, t, hq, D), _randn(gen, t, hkv, D), _randn(gen, t, hkv, D)
        st["pool"] = _pool(gen, nb, bs, hkv)
        st["src"] = torch.unique(page).to(torch.int32)
        st["dst"] = torch.arange(st["src"].numel(), dtype=torch.int32, device=DEV)
        st["k_blocks"] = torch.zeros(st["src"].numel(), bs, hkv, D, dtype=BF16, device=DEV)
        st["v_blocks"] = torch.zeros_like(st["k_blocks"])
    else:
        rows = n * c["new"] if c["kind"] == "window_prefill" else n
        st["q"] = (_randn(gen, rows, hq, D) * 1.5).to(BF16)
        if c["kind"] == "kv4_decode":
            st["pool"] = _pool(gen, nb, bs, hkv)
        else:
            st["k"], st["v"] = _randn(gen, nb, bs, hkv, D), _randn(gen, nb, bs, hkv, D)
        if c["kind"] == "window_prefill":
            st["starts"] = torch.arange(n + 1, dtype=torch.int32, device=DEV) * c["new"]
        st["out"] = torch.zeros(rows, hq, D, dtype=BF16 if c["kind"] == "window_prefill" else F32, device=DEV)
    if own:
        st["calls"] = _bind(st)
    return st


# ------------------------------------------------------- the framework's calls


def _bind(st):
    import paged_kv_cache_198_gb300 as tvl

    c = st["case"]
    if c["kind"] == "kv4_write":
        return [tvl.bind_kv4_write(st["k"], st["v"], st["pool"], st["slots"], q=st["q"],
                                   positions=st["positions"], rope_theta=500000.0),
                tvl.bind_kv4_expand_blocks(st["k_blocks"], st["v_blocks"], st["pool"], st["src"], st["dst"])]
    if c["kind"] == "kv4_decode":
        return [tvl.bind_kv4_attention_decode(st["out"], st["q"], st["pool"], st["tables"], st["ctx"], st["scale"],
                                              window=c["window"], sinks=c["sinks"])]
    if c["kind"] == "window_decode":
        return [tvl.bind_paged_attention_window_decode(st["out"], st["q"], st["k"], st["v"], st["tables"], st["ctx"],
                                                       st["scale"], c["window"], sinks=c["sinks"])]
    return [tvl.bind_paged_attention_window_prefill(st["out"], st["q"], st["starts"], st["k"], st["v"], st["tables"],
                                                    st["ctx"], st["scale"], c["new"], c["window"], sinks=c["sinks"])]


def run(state):
    kind = state["case"]["kind"]
    if own:
        for call in state["calls"]:
            call()
        if kind == "kv4_write":
            return {"q": state["q"], "k": state["k_blocks"], "v": state["v_blocks"]}
        return state["out"]
    if kind == "kv4_write":
        return _plain_write(state)
    if kind == "kv4_decode":
        return _plain_decode(state, *_plain_values(state["pool"]))
    if kind == "window_decode":
        return _plain_decode(state, state["k"], state["v"])
    return _plain_prefill(state)


# ------------------------------------------------------------ the plain forms


def _plain_rope(x, pos):
    """Angles in 64 bits (positions are far), the rotation in 32."""
    inv = 500000.0 ** (-torch.arange(D // 2, dtype=F64, device=x.device) * 2.0 / D)
    a = pos.to(F64)[:, None, None] * inv
    cos, sin = torch.cos(a).to(F32), torch.sin(a).to(F32)
    x0, x1 = x[..., :D // 2].to(F32), x[..., D // 2:].to(F32)
    return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], dim=-1).to(BF16)


def _plain_quantise(x):
    """Codes [T, Hkv, 32] in bytes and (s, z) [T, Hkv, 2] in bf16 of rows [T, Hkv, 64]."""
    x = x.to(F32)
    z = x.amin(dim=-1, keepdim=True)
    s = (x.amax(dim=-1, keepdim=True) - z) / torch.full_like(z, 15.0)   # a quotient, not a product with 1 / 15
    s = ((s.view(torch.int32) + 0xFFFF) & -0x10000).view(F32)     # up to the next bf16
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
    pool, slots = st["pool"], st["slots"].long()
    bs = st["case"]["bs"]
    st["q"].copy_(_plain_rope(st["q"], st["positions"]))
    page, sub, tok = slots // bs, slots % bs // 16, slots % 16
    for part, x in ((0, _plain_rope(st["k"], st["positions"])), (1, st["v"])):
        code, meta = _plain_quantise(x)
        pool[..., 512 * part:512 * part + 512].unflatten(-1, (16, 32))[page, sub, :, tok] = code
        pool[..., 1024 + 64 * part:1088 + 64 * part].unflatten(-1, (16, 4))[page, sub, :, tok] = meta.view(U8)
    k, v = _plain_values(pool[st["src"].long()])
    return {"q": st["q"], "k": k.to(BF16), "v": v.to(BF16)}


def _plain_decode(st, k, v):
    c, ctx = st["case"], st["ctx"].long()
    hkv, bs = c["hkv"], c["bs"]
    w, sinks = c["window"], c["sinks"]
    most = max(_visible(dict(c), x) for x in _lens(c))
    j = torch.arange(most, device=ctx.device)[None]
    first = (ctx - w).clamp(min=0)[:, None] if w else torch.zeros_like(ctx)[:, None]
    kept = first.clamp(max=sinks)                             # sinks ahead of the window
    pos = torch.where(j < kept, j, j - kept + first)
    seen = pos < ctx[:, None]
    pos = torch.where(seen, pos, 0)
    slot = torch.gather(st["tables"].long(), 1, pos // bs) * bs + pos % bs
    kk, vv = k.reshape(-1, hkv, D)[slot].to(F32), v.reshape(-1, hkv, D)[slot].to(F32)
    q = st["q"].to(F32).reshape(len(ctx), hkv, -1, D)
    s = (torch.einsum("shgd,snhd->shgn", q, kk) * st["scale"]).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(dim=-1, keepdim=True))
    o = torch.einsum("shgn,snhd->shgd", p, vv) / p.sum(dim=-1, keepdim=True)
    return o.reshape(len(ctx), c["hq"], D)


def _plain_prefill(st):
    c, ctx = st["case"], st["ctx"].long()
    n, hkv, bs, new = len(ctx), c["hkv"], c["bs"], c["new"]
    key = torch.arange(int(st["tables"].shape[1]) * bs, device=ctx.device)
    page = st["tables"].long().clamp(min=0)
    kk, vv = (x[page].reshape(n, -1, hkv, D).to(F32) for x in (st["k"], st["v"]))
    q = st["q"].to(F32).reshape(n, new, hkv, -1, D)
    at = (ctx[:, None] - new + torch.arange(new, device=ctx.device))[:, :, None]
    seen = key <= at
    if c["window"]:
        seen &= (key > at - c["window"]) | (key < c["sinks"])
    s = torch.einsum("sthgd,snhd->shgtn", q, kk).mul_(st["scale"]).masked_fill_(~seen[:, None, None], -math.inf)
    p = s.sub_(s.amax(dim=-1, keepdim=True)).exp_()
    o = torch.einsum("shgtn,snhd->sthgd", p.div_(p.sum(dim=-1, keepdim=True)), vv)
    return o.reshape(n * new, c["hq"], D).to(BF16)


# ---------------------------------------------------------------------- work


def work(case):
    c, lens = case, _lens(case)
    hq, hkv, n = c["hq"], c["hkv"], c["seqs"]
    if c["kind"] == "kv4_write":
        t, new, bs = n * c["new"], c["new"], c["bs"]
        # each new row read, each code written; the touched blocks read and expanded
        blocks = sum((x - 1) // bs - max(0, x - new) // bs + 1 for x in lens)
        return {"bytes": t * (2 * hkv * 128 + 2 * hq * 128 + hkv * 72 + 8) + blocks * bs * hkv * (72 + 256), "flops": 0}
    if c["kind"] == "window_prefill":
        pairs = sum(_visible(c, p + 1) for x in lens for p in range(x - c["new"], x))
        keys = sum(min(x, c["window"] + c["new"] - 1 + c["sinks"]) if c["window"] else x for x in lens)
        return {"bytes": keys * hkv * 256 + n * c["new"] * hq * 256, "flops": 4 * D * hq * pairs}
    seen = sum(_visible(c, x) for x in lens)
    row = 72 if c["kind"] == "kv4_decode" else 256
    return {"bytes": seen * hkv * row + n * hq * D * 6 + 4 * n + 4 * (seen // c["bs"]), "flops": 4 * D * hq * seen}


# -------------------------------------------------------------- in 64 bits


def _exact_values(pool, page, sub, head, tok, part):
    """One head's rows (index tensors of one shape) of a 4-bit cache, [..., 64]."""
    rec = pool[page, sub, head]
    byte = torch.gather(rec, -1, (512 * part + 32 * tok)[..., None] + torch.arange(32, device=rec.device))
    at = (1024 + 64 * part + 4 * tok)[..., None] + torch.arange(4, device=rec.device)
    sz = torch.gather(rec, -1, at).contiguous().view(BF16).to(F64)
    d = torch.arange(D, device=rec.device)
    code = (byte[..., d // 2].to(torch.int64) >> (4 * (d % 2))) & 15
    return sz[..., :1] * code.to(F64) + sz[..., 1:]


def _exact_rows(st, s, head, pos):
    """K and V rows of one head at positions `pos` of sequence s."""
    bs = st["case"]["bs"]
    page, off = st["tables"][s].long()[pos // bs], pos % bs
    if "pool" in st:
        return [_exact_values(st["pool"], page, off // 16, torch.full_like(page, head), off % 16, part) for part in (0, 1)]
    return [st[x][page, off, head].to(F64) for x in ("k", "v")]


def _exact_attention(st):
    c = st["case"]
    g, new, w = c["hq"] // c["hkv"], c.get("new", 1), c["window"]
    out = torch.zeros(c["seqs"], new, c["hq"], D, dtype=F64, device=DEV)
    q = st["q"].to(F64).reshape(c["seqs"], new, c["hq"], D)
    for s, n in enumerate(_lens(c)):
        first = max(0, n - new - w + 1) if w else 0
        keep = min(c["sinks"], first) if w else 0
        pos = torch.cat([torch.arange(0, keep, device=DEV), torch.arange(first, n, device=DEV)])
        for h in range(c["hkv"]):
            k, v = _exact_rows(st, s, h, pos)
            for r0 in range(0, new, 1024):
                r1 = min(new, r0 + 1024)
                at = torch.arange(n - new + r0, n - new + r1, device=DEV)[:, None]
                ok = pos <= at
                if w:
                    ok = ok & ((at - pos < w) | (pos < c["sinks"]))
                qq = q[s, r0:r1, h * g:(h + 1) * g].transpose(0, 1)
                p = torch.softmax((qq @ k.T * st["scale"]).masked_fill(~ok, -math.inf), dim=-1)
                out[s, r0:r1, h * g:(h + 1) * g] = (p @ v).transpose(0, 1)
    return out.reshape(-1, c["hq"], D)


def _exact_write(st):
    pos = st["positions"].to(F64)
    angle = pos[:, None] * torch.exp(-torch.arange(32, dtype=F64, device=DEV) / 32.0 * math.log(500000.0))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotate(x):
        z = torch.view_as_complex(torch.stack([x[..., :32], x[..., 32:]], dim=-1).to(F64)) * turn
        return torch.cat([z.real, z.imag], dim=-1)

    bs, src = st["case"]["bs"], st["src"].long()
    rows = src.numel() * bs
    place = torch.zeros(int(st["pool"].shape[0]), dtype=torch.int64, device=DEV)
    place[src] = torch.arange(src.numel(), device=DEV)
    slot = st["slots"].long()
    to = place[slot // bs] * bs + slot % bs
    got = {"q": rotate(st["q"])}
    r = torch.arange(rows, device=DEV)
    page, off = src[r // bs], r % bs
    # the rotated K is a bf16 row before it is quantised
    for name, part, x in (("k", 0, rotate(st["k"]).to(BF16).to(F64)), ("v", 1, st["v"].to(F64))):
        old = torch.stack([_exact_values(st["pool"], page, off // 16, torch.full_like(page, h), off % 16, part)
                           for h in range(st["case"]["hkv"])], dim=1)
        z, top = x.min(dim=-1, keepdim=True).values, x.max(dim=-1, keepdim=True).values
        m, e = torch.frexp((top - z) / torch.full_like(z, 15.0))
        two_e = ((e.to(torch.int64) + 1015) << 52).view(F64)  # 2 ** (e - 8), exactly
        s = torch.ceil(m * 256.0) * two_e                     # 8 significant bits, upwards
        code = torch.where(s > 0, torch.round((x - z) / s), 0.0).clamp(0, 15)
        old[to] = s * code + z
        got[name] = old.reshape(src.numel(), bs, -1, D)
    return got


def exact(case, seed):
    st = prepare({k: v for k, v in case.items() if k != "name"}, seed)
    return _exact_write(st) if case["kind"] == "kv4_write" else _exact_attention(st)
