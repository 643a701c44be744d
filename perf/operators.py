"""The paged quantized KV cache's operators, as they are measured: page tables
built on the GPU, tokens quantized into pages, tokens read back, and attention
of one or many new tokens per sequence over the pages.

A pool is uint8 [n_pages][kv heads][page tokens / 16][tile bytes]; a tile holds
16 tokens of one head: K codes, K scales, V codes, V scales (the byte order of
include/kvq.h).  Every case is a dict of plain values; sequence lengths come
from the case's own "lens_seed", values from the seed of prepare()."""
import math
import random

import numpy as np
import torch

own = False

D, NB = 128, 4
SCALE = 1.0 / math.sqrt(D)
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step of a full server: every request grows by a token
        dict(name="tables-decode", op="tables", n_seqs=256, page=64, len_hi=8192, grow=1.0, chunk_hi=1, release=0.0, lens_seed=1),
        # continuous batching under load: prompt chunks, decodes, idle and finished requests
        dict(name="tables-mixed", op="tables", n_seqs=1024, page=16, len_hi=16384, grow=0.7, chunk_hi=512, release=0.1, lens_seed=2),
        # one decode step of 64 requests, K and V taken out of a fused projection
        dict(name="append-decode", op="append", tokens=64, kv_heads=8, page=16, k="i8", v="q4", fused=True),
        # prompt chunks of a busy step
        dict(name="append-chunk", op="append", tokens=8192, kv_heads=8, page=64, k="i8", v="q8", fused=False),
        # a short prefix handed to a kernel that wants plain fp16
        dict(name="gather-prefix", op="gather", tokens=777, kv_heads=8, page=64, k="i8", v="q4", out="f16"),
        # a whole long context read back
        dict(name="gather-long", op="gather", tokens=131072, kv_heads=8, page=64, k="i8", v="q8", out="f32"),
        # the smallest decode: one request, one kv head
        dict(name="attn-tiny", op="attn", n_seqs=1, kv_heads=1, q_heads=4, len_lo=256, len_hi=256, chunks=0, q_lo=1, q_hi=1, page=64, k="i8", v="q8", out="f32", causal=True, lens_seed=3),
        # one request at the far end of a long context
        dict(name="attn-long", op="attn", n_seqs=1, kv_heads=8, q_heads=40, len_lo=131072, len_hi=131072, chunks=0, q_lo=1, q_hi=1, page=64, k="i8", v="q4", out="f16", causal=True, lens_seed=4),
        # a ragged decode batch
        dict(name="attn-batched", op="attn", n_seqs=64, kv_heads=8, q_heads=32, len_lo=1024, len_hi=32768, chunks=0, q_lo=1, q_hi=1, page=16, k="i8", v="q8", out="f32", causal=True, lens_seed=5),
        # four tokens per request to verify
        dict(name="attn-verify", op="attn", n_seqs=16, kv_heads=8, q_heads=64, len_lo=32768, len_hi=32768, chunks=16, q_lo=4, q_hi=4, page=64, k="i8", v="q4", out="f32", causal=True, lens_seed=6),
        # one chunk of a long prompt
        dict(name="attn-prefill", op="attn", n_seqs=1, kv_heads=8, q_heads=32, len_lo=32768, len_hi=32768, chunks=1, q_lo=512, q_hi=512, page=64, k="i8", v="q4", out="f16", causal=True, lens_seed=7),
        # prompt chunks and decodes in one ragged batch
        dict(name="attn-mixed", op="attn", n_seqs=44, kv_heads=8, q_heads=32, len_lo=500, len_hi=8192, chunks=4, q_lo=100, q_hi=512, page=16, k="i8", v="q8", out="f32", causal=True, idle=4, lens_seed=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "gather", "attn", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    ls = rng.randrange(1 << 30)
    if op == "tables":
        return dict(op=op, n_seqs=_log(rng, 1, 1024), page=page, len_hi=_log(rng, 16, 16384), grow=rng.uniform(0.3, 1.0),
                    chunk_hi=_log(rng, 1, 512), release=rng.choice([0.0, 0.1, 0.3]), lens_seed=ls)
    heads = rng.choice([1, 2, 4, 8])
    k, v = rng.choice(["i8", "i8", "i8", "f16"]), rng.choice(["q4", "q8"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=heads, page=page, k=k, v=v, fused=rng.random() < 0.5)
    if op == "gather":
        return dict(op=op, tokens=_log(rng, 1, 65536), kv_heads=heads, page=page, k=k, v=v, out=rng.choice(["f16", "f32"]))
    group = rng.choice([1, 3, 4, 5, 8])
    n = _log(rng, 1, 48)
    hi = _log(rng, 16, min(131072, 524288 // n))
    chunks = rng.choice([0, 0, n, max(1, n // 8)])
    q_hi = _log(rng, 2, max(2, min(hi, 512, (1 << 28) // (n * hi * heads * group)))) if chunks else 1
    return dict(op=op, n_seqs=n, kv_heads=heads, q_heads=heads * group, len_lo=max(1, hi // rng.choice([1, 4, 16])), len_hi=hi,
                chunks=chunks, idle=n // 8 if chunks < n else 0, q_lo=max(1, q_hi // 2), q_hi=q_hi, page=page, k="i8" if chunks else k, v=v,
                out=rng.choice(["f16", "f32"]), causal=rng.random() < 0.8, lens_seed=ls)


def _shape(case):
    """Sequence lengths (with the new tokens) and new tokens of an attn case."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["n_seqs"])]
    newt = [r.randint(case["q_lo"], case["q_hi"]) if b < case["chunks"] else 1 for b in range(case["n_seqs"])]
    newt = [min(a, b) for a, b in zip(newt, lens)]
    for b in range(case.get("idle", 0)):  # places of the batch that no request holds
        lens[-1 - b] = newt[-1 - b] = 0
    order = list(range(case["n_seqs"]))
    r.shuffle(order)
    return [lens[b] for b in order], [newt[b] for b in order]


def _requests(case):
    """Held tokens and requested growth (-1: finished) of a tables case."""
    r = random.Random(case["lens_seed"])
    lens, newt = [], []
    for _ in range(case["n_seqs"]):
        lens.append(r.randint(0, case["len_hi"]))
        x = r.random()
        newt.append(-1 if x < case["release"] else 0 if r.random() > case["grow"] else r.choice([1, r.randint(1, case["chunk_hi"])]))
    return lens, newt


# ----------------------------------------------------------------- layout --
def _tile_bytes(k, v):
    return (2048 + 128 if k == "i8" else 4096) + (1024 if v == "q4" else 2048) + 128


_maps_kept = {}


def _maps(k, v):
    """Byte offsets in a tile of token u: K bytes (or fp16 halves) [16, 128],
    K scales [16, 4], V bytes [16, 64 or 128], V scales [16, 4]."""
    if (k, v) in _maps_kept:
        return _maps_kept[(k, v)]
    u = torch.arange(16)[:, None]
    sub, gu, cu, e = u // 8, u % 8, (u % 8) // 2, u % 2
    j = torch.arange(128)[None, :]
    if k == "i8":
        ko = ((2 * sub + j // 64) * 32 + 4 * gu + (j % 32) // 8) * 16 + 8 * ((j // 32) % 2) + j % 8
        base = 2048
    else:
        ko = (j // 16) * 512 + (4 * gu + (j % 8) // 2) * 16 + 4 * (sub + 2 * ((j % 16) // 8)) + 2 * (j % 2)
        base = 4096
    b = torch.arange(4)[None, :]
    so = 2 * ((sub * 4 + cu) * 8 + b * 2 + e)
    kso = base + so if k == "i8" else None
    base += 128 if k == "i8" else 0
    if v == "q4":
        jv = torch.arange(64)[None, :]
        vo = (sub * 32 + 4 * ((jv % 16) // 2) + cu) * 16 + 4 * (jv // 16) + 2 * e + jv % 2
        vb = 1024
    else:
        vo = ((2 * sub + j // 64) * 32 + 4 * ((j % 32) // 4) + cu) * 16 + 8 * ((j // 32) % 2) + 4 * ((j % 4) // 2) + 2 * (j % 2) + e
        vb = 2048
    got = [None if x is None else x.to(DEV) for x in (ko, kso, base + vo, base + vb + so)]
    _maps_kept[(k, v)] = got
    return got


def _away(x):
    """Nearest whole number, halves away from zero."""
    a = x.abs()
    f = a.floor()
    return torch.sign(x) * (f + (a - f >= 0.5).to(x.dtype))


def _quant8(x):
    """int8 rule on 32-blocks: fp16 scale [..., 4], codes [..., 128] (float)."""
    y = x.float().unflatten(-1, (NB, 32))
    s = (y.abs().amax(-1, keepdim=True) / 127.0).half()
    c = torch.where(s == 0, torch.zeros_like(y), _away(y / s.float()).clamp(-127, 127))
    return s.squeeze(-1), c.flatten(-2)


def _quant4(x):
    y = x.float().unflatten(-1, (NB, 32))
    d = (y.abs().amax(-1, keepdim=True) * 0.125).half()
    c = torch.where(d == 0, torch.full_like(y, 8.0), (_away(y / d.float()) + 8.0).clamp(0, 15))
    return d.squeeze(-1), c.flatten(-2)


def _put(rows, off, vals):
    rows.scatter_(-1, off.expand(vals.shape), vals)


def _pack(rows, u, k16, v16, k, v):
    """Writes tokens into copies of their tiles: rows uint8 [T, H, tile bytes],
    u [T] the token's place in its tile; returns the byte offsets written."""
    ko, kso, vo, vso = _maps(k, v)
    offs, vals = [], []

    def bytes2(o, x):  # 2-byte values at byte offsets o
        offs.extend([o[u][:, None, :], o[u][:, None, :] + 1])
        b = x.contiguous().view(torch.uint8).unflatten(-1, (-1, 2))
        vals.extend([b[..., 0], b[..., 1]])

    if k == "i8":
        s, c = _quant8(k16)
        offs.append(ko[u][:, None, :])
        vals.append((c + 128).to(torch.uint8))
        bytes2(kso, s)
    else:
        bytes2(ko, k16)
    if v == "q8":
        s, c = _quant8(v16)
        vals.append((c + 128).to(torch.uint8))
    else:
        s, c = _quant4(v16)
        c = c.unflatten(-1, (NB, 2, 16))
        vals.append((c[..., 0, :] + 16 * c[..., 1, :]).flatten(-2).to(torch.uint8))
    offs.append(vo[u][:, None, :])
    bytes2(vso, s)
    H = rows.shape[1]
    return torch.cat([o.expand(-1, H, -1) for o in offs], -1), torch.cat(vals, -1)


def _fill_pool(gen, n_pages, H, page, k, v, outliers=True):
    """A pool whose every token was quantized from N(0, 1) values, four channels
    of each head ten times as large."""
    tb = _tile_bytes(k, v)
    pool = torch.empty((n_pages, H, page // 16, tb), dtype=torch.uint8, device=DEV)
    amp = torch.ones((H, D), device=DEV)
    if outliers:
        amp.scatter_(1, torch.rand((H, D), device=DEV, generator=gen).topk(4, dim=1).indices, 10.0)
    step = max(1, (1 << 25) // (H * page * D))
    u = torch.arange(page, device=DEV) % 16
    for p0 in range(0, n_pages, step):
        n = min(step, n_pages - p0)
        kv = torch.randn((2, n * page, H, D), device=DEV, generator=gen)
        kv = (kv * amp).half()
        uu = u.repeat(n)
        off, val = _pack(pool[:1, :, 0].expand(n * page, H, tb), uu, kv[0], kv[1], k, v)
        # token (page, tile, u) of head h: into its tile's bytes
        tile = pool[p0:p0 + n]
        off = off.view(n, page // 16, 16, H, -1).permute(0, 3, 1, 2, 4).reshape(n, H, page // 16, -1)
        val = val.view(n, page // 16, 16, H, -1).permute(0, 3, 1, 2, 4).reshape(n, H, page // 16, -1)
        tile.scatter_(-1, off, val)
    return pool


# ---------------------------------------------------------------- prepare --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7fffffff)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "tables":
        return _prepare_tables(case, g, st)
    page, H, k, v = case["page"], case["kv_heads"], case["k"], case["v"]
    if case["op"] in ("append", "gather"):
        T = case["tokens"]
        n_pages = (T + page - 1) // page + 3
        st["pool"] = _fill_pool(g, n_pages, H, page, k, v)
        st["slots"] = _some_slots(g, T, n_pages, page, scattered=case["op"] == "append" and T <= 256)
        if case["op"] == "append":
            if case.get("fused"):  # K and V as columns of one projection's output, query heads before them
                x = torch.randn((T, (4 + 2) * H, D), device=DEV, generator=g).half()
                st["k16"], st["v16"] = x[:, 4 * H:5 * H], x[:, 5 * H:]
            else:
                st["k16"] = torch.randn((T, H, D), device=DEV, generator=g).half()
                st["v16"] = torch.randn((T, H, D), device=DEV, generator=g).half()
        dt = torch.float16 if case.get("out") == "f16" else torch.float32
        st["k_out"], st["v_out"] = (torch.zeros((T, H, D), dtype=dt, device=DEV) for _ in range(2))
        return st
    lens, newt = _shape(case)
    blocks = [(n + page - 1) // page for n in lens]
    n_pages = sum(blocks) + 5
    st["pool"] = _fill_pool(g, n_pages, H, page, k, v)
    ids = torch.randperm(n_pages, device=DEV, generator=g).int()
    bt = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = ids[at:at + n]
        at += n
    T = sum(newt)
    st["block_table"] = bt
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["q_start"] = torch.tensor([0] + list(np.cumsum(newt)), dtype=torch.int32, device=DEV)
    st["max_q"], st["max_len"] = max(newt), max(lens)
    st["q16"] = torch.randn((T, case["q_heads"], D), device=DEV, generator=g).half()
    dt = torch.float16 if case["out"] == "f16" else torch.float32
    st["out"] = torch.zeros((T, case["q_heads"], D), dtype=dt, device=DEV)
    st["lse"] = torch.zeros((T, case["q_heads"]), dtype=torch.float32, device=DEV)
    return st


def _some_slots(g, T, n_pages, page, scattered):
    if scattered:  # one token of each of T requests
        return torch.randperm(n_pages * page, device=DEV, generator=g)[:T].int()
    order = torch.randperm(n_pages, device=DEV, generator=g)
    pos = torch.arange(T, device=DEV) + page // 2
    return (order[pos // page] * page + pos % page).int()


def _prepare_tables(case, g, st):
    lens, newt = _requests(case)
    page, B = case["page"], case["n_seqs"]
    have = [(n + page - 1) // page for n in lens]
    most = (case["len_hi"] + case["chunk_hi"] + page - 1) // page
    T = sum(max(0, n) for n in newt)
    need = sum((a + n + page - 1) // page - h for a, n, h in zip(lens, newt, have) if n > 0)
    n_pages = sum(have) + need + 7
    ids = torch.randperm(n_pages, device=DEV, generator=g).int()
    bt = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(have):
        bt[b, :n] = ids[at:at + n]
        at += n
    n_free = n_pages - at
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    free[:n_free] = ids[at:]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def buf(n):
        return torch.zeros(n, dtype=torch.int32, device=DEV)

    st.update(n_pages=n_pages, lens=i32(lens), n_new=i32(newt), block_table=bt, free=free, n_free=i32([n_free]),
              lens_out=buf(B), n_free_out=buf(1), q_start=buf(B + 1), slots=buf(max(1, T)), status=buf(B), tokens=T)
    return st


# -------------------------------------------------------------------- run --
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "tables":
        return _plain_tables(state)
    if op == "append":
        _plain_append(state)
    if op in ("append", "gather"):
        k, v = _plain_read(state["pool"], state["slots"], state["case"])
        dt = state["k_out"].dtype
        return {"k": k.to(dt), "v": v.to(dt)}
    return _plain_attn(state)


def _own(state, op):
    """The calls a serving loop makes; the prepared calls are kept as it keeps them."""
    from quantized_kv_cache_03_gb300 import kvq
    call = state.get("call")
    if call is None:
        call = state["call"] = _own_calls(kvq, state, op)
    for c in call:
        c()
    if op == "tables":
        return {"block_table": state["block_table"], "slots": state["slots"], "q_start": state["q_start"],
                "lens": state["lens_out"], "free": state["free"], "n_free": state["n_free_out"], "status": state["status"]}
    if op in ("append", "gather"):
        return {"k": state["k_out"], "v": state["v_out"]}
    return {"out": state["out"], "lse": state["lse"]}


def _own_calls(kvq, s, op):
    case = s["case"]
    if op == "tables":
        return [kvq.PageTablesCall(case["page"], s["n_pages"], s["lens"], s["n_new"], s["free"], s["n_free"], s["block_table"],
                                   s["lens_out"], s["n_free_out"], s["q_start"], s["slots"], s["status"])]
    pool = kvq.PagePool(s["pool"].shape[0], case["page"], case["kv_heads"], kvq.V_Q4_0 if case["v"] == "q4" else kvq.V_Q8_0,
                        k_type=kvq.K_I8 if case["k"] == "i8" else kvq.K_F16, data=s["pool"])
    if op in ("append", "gather"):
        gather = kvq.PagedGatherCall(pool, s["slots"], s["k_out"], s["v_out"])
        return [gather] if op == "gather" else [kvq.PagedAppendCall(pool, s["k16"], s["v16"], s["slots"]), gather]
    return [kvq.PagedAttnCall(pool, s["q16"], s["q_start"], s["max_q"], s["lens"], s["block_table"], case["causal"], SCALE,
                              s["out"], s["lse"])]


def _plain_tables(s):
    case = s["case"]
    P, B = case["page"], case["n_seqs"]
    lens, newt, bt, free = s["lens"].long(), s["n_new"].long(), s["block_table"].clone(), s["free"].clone()
    n_free, most, T = s["n_free"].long(), bt.shape[1], s["tokens"]
    have = (lens + P - 1) // P
    grow = newt.clamp(min=0)
    q_start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), grow.cumsum(0)])
    fits = ((lens + grow) <= most * P) & (q_start[1:] <= T)
    need = torch.where((newt > 0) & fits, (lens + grow + P - 1) // P - have, torch.zeros_like(lens))
    back = torch.where(newt < 0, have, torch.zeros_like(have))
    # the stack: free pages, then those of finished sequences in order
    cols = torch.arange(most, device=DEV)[None, :]
    v = torch.arange(free.numel(), device=DEV)
    ends = back.cumsum(0)
    avail = n_free + ends[-1]
    of = torch.searchsorted(ends, v - n_free, right=True).clamp(max=B - 1)
    col = (v - n_free - (ends[of] - back[of])).clamp(0, most - 1)
    stack = torch.where(v < n_free, free, bt[of, col])
    last = need.cumsum(0)
    granted = fits & ((need == 0) | (last <= avail))
    first = last - need
    pos = cols - have[:, None]
    takes = granted[:, None] & (pos >= 0) & (pos < need[:, None])
    at = (avail - 1 - first[:, None] - pos).clamp(0, free.numel() - 1)
    bt = torch.where(takes, stack[at], bt)
    n_out = avail - torch.where(granted, need, torch.zeros_like(need)).sum()
    free = torch.where((v >= n_free) & (v < n_out), stack, free)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(q_start[1:], t, right=True)
    p = lens[b] + t - q_start[b]
    slots = torch.where(granted[b], bt[b, p // P].long() * P + p % P, torch.full_like(p, -1))
    lens_out = torch.where(newt < 0, torch.zeros_like(lens), lens + torch.where(granted, grow, torch.zeros_like(grow)))
    status = torch.where((newt > 0) & ~fits, 2, torch.where((newt > 0) & ~granted, 1, 0))
    return {"block_table": bt, "slots": slots.int() if T else s["slots"], "q_start": q_start.int(), "lens": lens_out.int(), "free": free,
            "n_free": n_out.int().reshape(1), "status": status.int()}


def _plain_append(s):
    case, slots = s["case"], s["slots"].long()
    page, off = slots // case["page"], slots % case["page"]
    pool, u = s["pool"], off % 16
    rows = pool[page, :, off // 16]
    o, val = _pack(rows, u, s["k16"], s["v16"], case["k"], case["v"])
    H, tb = rows.shape[1], rows.shape[2]
    base = ((page[:, None] * H + torch.arange(H, device=DEV)) * (case["page"] // 16) + (off // 16)[:, None]) * tb
    pool.view(-1)[(base[..., None] + o).reshape(-1)] = val.reshape(-1)


def _plain_read(pool, slots, case):
    """Dequantized K and V, fp32 [tokens, kv heads, 128], of the listed slots."""
    slots = slots.long()
    page, off = slots // case["page"], slots % case["page"]
    rows, u = pool[page, :, off // 16], off % 16
    ko, kso, vo, vso = _maps(case["k"], case["v"])
    H = rows.shape[1]

    def take(o):
        return rows.gather(-1, o[u][:, None, :].expand(-1, H, -1))

    def half(o):
        o2 = torch.stack([o, o + 1], -1).flatten(-2)
        return take(o2).view(torch.float16).float()

    if case["k"] == "i8":
        k = (take(ko).float() - 128.0).unflatten(-1, (NB, 32)) * half(kso)[..., None]
        k = k.flatten(-2)
    else:
        k = half(ko)
    c = take(vo)
    if case["v"] == "q8":
        c = c.float() - 128.0
    else:
        c = c.unflatten(-1, (NB, 16))
        c = torch.cat([(c & 15).float(), (c >> 4).float()], -1).flatten(-2) - 8.0
    v = (c.unflatten(-1, (NB, 32)) * half(vso)[..., None]).flatten(-2)
    return k, v


def _plain_attn(s):
    case = s["case"]
    P, H, Hq, B = case["page"], case["kv_heads"], case["q_heads"], case["n_seqs"]
    G, L, Q = Hq // H, s["max_len"], s["max_q"]
    lens, qs = s["lens"].long(), s["q_start"].long()
    newt = qs[1:] - qs[:-1]
    pos = torch.arange(L, device=DEV)
    slots = s["block_table"].long()[:, pos // P].clamp(min=0) * P + pos % P
    k, v = _plain_read(s["pool"], slots.reshape(-1), case)
    k, v = (x.view(B, L, H, D).transpose(1, 2) for x in (k, v))
    if case["k"] == "i8":
        sq, cq = _quant8(s["q16"])
        q = (cq.unflatten(-1, (NB, 32)) * sq.float()[..., None]).flatten(-2)
    else:
        q = s["q16"].float()
    i = torch.arange(Q, device=DEV)
    row = (qs[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qp = q[row].view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    x = (torch.matmul(qp, k.transpose(-1, -2)) * SCALE).view(B, H, Q, G, L)
    lim = lens[:, None] - newt[:, None] + i if case["causal"] else (lens[:, None] - 1).expand(B, Q)
    seen = (pos <= lim[..., None]) & (pos < lens[:, None, None])
    x = x.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H, Q * G, L), v).view(B, H, Q, G, D) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    t = torch.arange(q.shape[0], device=DEV)
    b = torch.searchsorted(qs[1:], t, right=True)
    j = t - qs[b]
    o = o.permute(0, 2, 1, 3, 4)[b, j].reshape(-1, Hq, D)
    lse = lse.permute(0, 2, 1, 3)[b, j].reshape(-1, Hq)
    return {"out": o.to(s["out"].dtype), "lse": lse}


# ------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "tables":
        lens, newt = _requests(case)
        P = case["page"]
        T = sum(max(0, n) for n in newt)
        new = sum((a + n + P - 1) // P - (a + P - 1) // P for a, n in zip(lens, newt) if n > 0)
        back = sum((a + P - 1) // P for a, n in zip(lens, newt) if n < 0)
        return {"bytes": 4.0 * (2 * len(lens) + 3 * len(lens) + T + 2 * new + 2 * back + 2), "flops": 0.0}
    per = _tile_bytes(case["k"], case["v"]) / 16 * case["kv_heads"]
    if op in ("append", "gather"):
        T, vals = case["tokens"], case["tokens"] * case["kv_heads"] * D * 2
        if op == "gather":
            return {"bytes": T * (per + 4) + vals * (2 if case["out"] == "f16" else 4), "flops": float(vals)}
        return {"bytes": T * (2 * per + 8) + vals * 2 + vals * 4, "flops": 3.0 * vals}
    lens, newt = _shape(case)
    seen = sum(n * (L - n) + n * (n + 1) // 2 if case["causal"] else n * L for L, n in zip(lens, newt))
    T = sum(newt)
    out = T * case["q_heads"] * (D * (2 if case["out"] == "f16" else 4) + 4)
    table = 4 * sum((L + case["page"] - 1) // case["page"] for L in lens)
    return {"bytes": sum(lens) * per + T * case["q_heads"] * D * 2 + out + table, "flops": 4.0 * D * case["q_heads"] * seen}


# ------------------------------------------------------------------ exact --
def _tile_values(tiles, k, v):
    """[N, tile bytes] uint8 -> K and V as float64 [N, 16, 128], read the way a
    warp reads a tile: 16-byte words of lane 4g + c."""
    N = tiles.shape[0]
    if k == "f16":
        w = tiles[:, :4096].contiguous().view(torch.float16).double().view(N, 8, 8, 4, 2, 2, 2)
        K = w.permute(0, 5, 2, 1, 4, 3, 6).reshape(N, 16, D)    # from: k16 step, g, c, half of the step, token half, pair
        at = 4096
    else:
        w = tiles[:, :2048].double().view(N, 2, 2, 8, 4, 2, 8) - 128.0     # sub, block pair, g, c, block, code
        K = w.permute(0, 1, 3, 2, 5, 4, 6).reshape(N, 16, D) * _tile_scales(tiles[:, 2048:2176])
        at = 2176
    if v == "q4":
        w = tiles[:, at:at + 1024].view(N, 2, 8, 4, 4, 2, 2)     # sub, g, c, block, token of the pair, byte of the pair
        w = w.permute(0, 1, 3, 5, 4, 2, 6).reshape(N, 16, 4, 16)
        V = torch.cat([w % 16, w // 16], -1).double().reshape(N, 16, D) - 8.0
        at += 1024
    else:
        w = tiles[:, at:at + 2048].double().view(N, 2, 2, 8, 4, 2, 2, 2, 2) - 128.0
        # sub, block pair, g, c, block, dim pair, dim, token of the pair
        V = w.permute(0, 1, 4, 8, 2, 5, 3, 6, 7).reshape(N, 16, D)
        at += 2048
    return K, V * _tile_scales(tiles[:, at:at + 128])


def _tile_scales(raw):
    s = raw.contiguous().view(torch.float16).double().view(-1, 2, 4, 4, 2)    # sub, c, block, token of the pair
    return s.permute(0, 1, 2, 4, 3).reshape(-1, 16, 4).repeat_interleave(32, dim=-1)


def _round_blocks(x, top, div, shift, low, high, zero):
    """One 32-block rule in 64 bits with its fp16 scale: the value each element stands for."""
    y = x.astype(np.float64).reshape(x.shape[:-1] + (NB, 32))
    s = (np.abs(y).max(-1, keepdims=True).astype(np.float32) / np.float32(div)).astype(np.float16).astype(np.float64)
    r = y / np.where(s == 0, 1.0, s)
    c = np.where(r < 0, np.ceil(r - 0.5), np.floor(r + 0.5)) + shift
    c = np.where(s == 0, zero, np.clip(c, low, high)) - shift
    return (c * s).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    k, v, P, H = case["k"], case["v"], case["page"], case["kv_heads"]
    if case["op"] == "append":
        k16, v16 = s["k16"].cpu().numpy(), s["v16"].cpu().numpy()
        kk = k16.astype(np.float64) if k == "f16" else _round_blocks(k16, 127, 127.0, 0, -127, 127, 0)
        vv = _round_blocks(v16, 127, 127.0, 0, -127, 127, 0) if v == "q8" else _round_blocks(v16, 8, 8.0, 8, 0, 15, 8)
        return {"k": torch.from_numpy(kk), "v": torch.from_numpy(vv)}
    if case["op"] == "gather":
        sl, pool = s["slots"].long(), s["pool"]
        K, V = _tile_values(pool.view(-1, pool.shape[-1]), k, v)
        K, V = (x.view(pool.shape[0], H, P, D)[sl // P, :, sl % P] for x in (K, V))
        return {"k": K, "v": V}
    lens, newt = _shape(case)
    G = case["q_heads"] // H
    q16 = s["q16"].cpu().numpy()
    q = q16.astype(np.float64) if k == "f16" else _round_blocks(q16, 127, 127.0, 0, -127, 127, 0)
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (L, n) in enumerate(zip(lens, newt)):
        if n == 0:
            continue
        tiles = s["pool"][s["block_table"][b, :(L + P - 1) // P].long()]
        K, V = _tile_values(tiles.view(-1, tiles.shape[-1]), k, v)
        for h in range(H):
            kh, vh = (x.view(-1, H, P, D)[:, h].reshape(-1, D)[:L] for x in (K, V))
            qh = torch.from_numpy(np.ascontiguousarray(q[t0:t0 + n, h * G:(h + 1) * G])).to(DEV)
            x = torch.einsum("igd,ld->igl", qh, kh) * SCALE
            if case["causal"]:
                far = torch.arange(L, device=DEV)[None, :] > (L - n + torch.arange(n, device=DEV))[:, None]
                x = x.masked_fill(far[:, None, :], -math.inf)
            z = torch.logsumexp(x, -1)
            out[t0:t0 + n, h * G:(h + 1) * G] = torch.einsum("igl,ld->igd", torch.exp(x - z[..., None]), vh)
            lse[t0:t0 + n, h * G:(h + 1) * G] = z
        t0 += n
    return {"out": out, "lse": lse}
