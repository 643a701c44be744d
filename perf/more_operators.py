"""What surrounds the paged quantized cache's append and attention, as it is
measured: new tokens on their way in (heads normalized, positions rotated, keys
and values quantized into pages), sequences forked, cut back and ended by their
page tables, pages copied in every layer's pool, and held tokens moved and
turned to other positions.

A pool is uint8 [n_pages][kv heads][page tokens / 16][tile bytes]; a tile holds
16 tokens of one head: K codes, K scales, V codes, V scales (the byte order of
include/kvq.h).  Every case is a dict of plain values; lengths, parents and
places come from the case's own "lens_seed", values and page numbers from the
seed of prepare()."""
import math
import random

import numpy as np
import torch

own = False

D, NB = 128, 4
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token of one small request, its rotated key left as fp16 for a cache in segments
        dict(name="qkv-tiny", op="qkv", tokens=1, n_seqs=1, q_heads=4, kv_heads=1, n_rot=128, layout="pairs", scaling="none", norm=False, to="plain", derived=False, fused=False, page=64, k="i8", v="q8", pos_hi=256, lens_seed=1),
        # one decode step of 64 requests, positions worked out from the step's lengths
        dict(name="qkv-decode", op="qkv", tokens=64, n_seqs=64, q_heads=32, kv_heads=8, n_rot=128, layout="half", scaling="turns", norm=True, to="pages", derived=True, fused=True, page=16, k="i8", v="q8", pos_hi=32768, lens_seed=2),
        # a ragged step whose heads are rotated in part, F16 K, far positions of a stretched context
        dict(name="qkv-partial", op="qkv", tokens=777, n_seqs=9, q_heads=64, kv_heads=8, n_rot=64, layout="pairs", scaling="index", norm=False, to="pages", derived=True, fused=False, page=64, k="f16", v="q4", pos_hi=131072, lens_seed=3),
        # prompt chunks of a busy step
        dict(name="qkv-prompt", op="qkv", tokens=8192, n_seqs=20, q_heads=40, kv_heads=8, n_rot=128, layout="half", scaling="linear", norm=True, to="pages", derived=False, fused=True, page=64, k="i8", v="q4", pos_hi=32768, lens_seed=4),
        # tokens of a verified tree kept: the accepted ones close ranks
        dict(name="move-accept", op="move", kind="accept", tokens=64, kv_heads=8, page=16, k="i8", v="q4", n_rot=0, layout="half", gap=0, lens_seed=5),
        # a context that lets go of 100 tokens in its middle: the rest moves up and turns back
        dict(name="move-shift", op="move", kind="shift", tokens=8092, kv_heads=8, page=64, k="i8", v="q8", n_rot=128, layout="half", gap=100, lens_seed=6),
        # whole pages let go: the other keys of a long context turn where they lie
        dict(name="move-turn", op="move", kind="turn", tokens=131072, kv_heads=8, page=64, k="i8", v="q4", n_rot=128, layout="half", gap=512, lens_seed=7),
        # one step of 64 searches with 4 beams each
        dict(name="fork-beams", op="fork", n_seqs=256, group=4, page=64, len_hi=8192, swap=0.6, cut=0.0, end=0.0, lens_seed=8),
        # a server's step: requests end, drop rejected tokens, start from others' prefixes
        dict(name="fork-server", op="fork", n_seqs=1024, group=2, page=16, len_hi=16384, swap=0.2, cut=0.3, end=0.1, lens_seed=9),
        # the shared last pages of one beam step, in each of 32 layers
        dict(name="copy-beams", op="copy", n_copies=256, pools=32, share=0.4, kv_heads=8, page=16, k="i8", v="q4", held=True, lens_seed=10),
        # one page in one small pool
        dict(name="copy-one", op="copy", n_copies=1, pools=1, share=1.0, kv_heads=1, page=64, k="i8", v="q8", held=False, lens_seed=11),
        # a context of 131072 tokens copied whole
        dict(name="copy-context", op="copy", n_copies=2048, pools=1, share=1.0, kv_heads=8, page=64, k="i8", v="q8", held=False, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qkv", "qkv", "qkv", "move", "move", "fork", "fork", "copy"])
    page = rng.choice([16, 32, 64, 128])
    ls = rng.randrange(1 << 30)
    if op == "fork":
        group = rng.choice([1, 2, 4, 8])
        return dict(op=op, n_seqs=group * _log(rng, 1, 1024 // group), group=group, page=page, len_hi=_log(rng, 16, 16384), swap=rng.choice([0.0, 0.3, 0.8]),
                    cut=rng.choice([0.0, 0.3]), end=rng.choice([0.0, 0.1, 0.5]), lens_seed=ls)
    heads = rng.choice([1, 2, 4, 8])
    k, v = rng.choice(["i8", "i8", "i8", "f16"]), rng.choice(["q4", "q8"])
    if op == "copy":
        n = _log(rng, 1, 2048 * 64 // page)
        pools = max(1, min(rng.choice([1, 5, 32]), (2048 * 64 // page) // n))
        return dict(op=op, n_copies=n, pools=pools, share=rng.choice([1.0, 0.5]), kv_heads=heads, page=page, k=k, v=v, held=rng.random() < 0.5, lens_seed=ls)
    n_rot = rng.choice([128, 128, 64, 32, 96, 40])
    layout = rng.choice(["half", "pairs"])
    if op == "move":
        kind = rng.choice(["accept", "shift", "turn"])
        return dict(op=op, kind=kind, tokens=_log(rng, 1, 65536), kv_heads=heads, page=page, k=k, v=v, n_rot=0 if kind == "accept" else n_rot, layout=layout,
                    gap=0 if kind == "accept" else _log(rng, 1, 4096), lens_seed=ls)
    tokens = _log(rng, 1, 8192)
    return dict(op=op, tokens=tokens, n_seqs=_log(rng, 1, min(tokens, 256)), q_heads=heads * rng.choice([1, 3, 4, 5]), kv_heads=heads, n_rot=rng.choice([n_rot, 0]) if rng.random() < 0.2 else n_rot,
                layout=layout, scaling=rng.choice(["none", "linear", "base", "index", "turns"]), norm=rng.random() < 0.5, to=rng.choice(["pages", "pages", "plain"]),
                derived=rng.random() < 0.5, fused=rng.random() < 0.5, page=page, k=k, v=v, pos_hi=_log(rng, 256, 131072), lens_seed=ls)


def _step(case):
    """Lengths (new tokens counted) and new tokens of a qkv case's sequences."""
    r = random.Random(case["lens_seed"])
    B, T = case["n_seqs"], case["tokens"]
    cuts = sorted(r.sample(range(1, T), B - 1)) if B > 1 else []
    new = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    return [n + r.randint(0, case["pos_hi"]) for n in new], new


def _frequencies(case):
    """Angles per position (float64) of a case's rotated pairs, and the factor on them."""
    n, kind = case["n_rot"], case.get("scaling", "none")
    base, factor, original = 10000.0, 8.0, 4096.0
    i = np.arange(n // 2, dtype=np.float64)
    if kind == "base":
        base = base * factor ** (n / (n - 2.0)) if n else base
    f = base ** (-2.0 * i / max(n, 1))
    if kind == "linear":
        return f / factor, 1.0
    if kind == "index":   # pairs that turn often keep their rate, those that never turn once are slowed, by the pair's number between
        at = [n * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        w = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / factor * w + f * (1 - w), 0.1 * math.log(factor) + 1.0
    if kind == "turns":   # the same by how often the pair turns within the original context
        w = np.clip((original * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0, 1)
        return f / factor * (1 - w) + f * w, 1.0
    return f, 1.0


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


def _two(o):
    """Offsets of both bytes of 2-byte values."""
    return torch.stack([o, o + 1], -1).flatten(-2)


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


def _half_bytes(x):
    return x.contiguous().view(torch.uint8)


def _k_bytes(k16, k):
    """K bytes of fp16 rows in the maps' order: codes and scales, or the values."""
    if k == "f16":
        return [_half_bytes(k16)]
    s, c = _quant8(k16)
    return [(c + 128).to(torch.uint8), _half_bytes(s)]


def _v_bytes(v16, v):
    if v == "q8":
        s, c = _quant8(v16)
        return [(c + 128).to(torch.uint8), _half_bytes(s)]
    s, c = _quant4(v16)
    c = c.unflatten(-1, (NB, 2, 16))
    return [(c[..., 0, :] + 16 * c[..., 1, :]).flatten(-2).to(torch.uint8), _half_bytes(s)]


def _offsets(k, v):
    """[16, bytes of a token] tile offsets of the bytes of _k_bytes and _v_bytes, and how many are K's."""
    ko, kso, vo, vso = _maps(k, v)
    ks = [_two(ko)] if k == "f16" else [ko, _two(kso)]
    ks = torch.cat(ks, -1)
    return torch.cat([ks, vo, _two(vso)], -1), ks.shape[1]


def _addresses(pool, slots, case):
    """Byte addresses [tokens, heads, bytes] of the listed slots' tokens in the pool."""
    P, (_, H, tiles, tb) = case["page"], pool.shape
    page, off = slots // P, slots % P
    o = _offsets(case["k"], case["v"])[0]
    base = ((page[:, None] * H + torch.arange(H, device=DEV)) * tiles + (off // 16)[:, None]) * tb
    return base[..., None] + o[off % 16][:, None, :]


def _read_values(b, case):
    """fp32 K and V of token bytes [tokens, heads, bytes] in the maps' order."""
    k, v = case["k"], case["v"]
    n = _offsets(k, v)[1]
    if k == "i8":
        s = b[..., 128:136].contiguous().view(torch.float16).float()
        kk = ((b[..., :128].float() - 128.0).unflatten(-1, (NB, 32)) * s[..., None]).flatten(-2)
    else:
        kk = b[..., :256].contiguous().view(torch.float16).float()
    vb = b[..., n:]
    s = vb[..., -8:].contiguous().view(torch.float16).float()
    c = vb[..., :-8]
    if v == "q8":
        c = c.float() - 128.0
    else:
        c = c.unflatten(-1, (NB, 16))
        c = torch.cat([(c & 15).float(), (c >> 4).float()], -1).flatten(-2) - 8.0
    return kk, (c.unflatten(-1, (NB, 32)) * s[..., None]).flatten(-2)


def _fill_pool(gen, n_pages, H, page, k, v):
    """A pool whose every token was quantized from N(0, 1) values, four channels
    of each head ten times as large."""
    tb = _tile_bytes(k, v)
    pool = torch.empty((n_pages, H, page // 16, tb), dtype=torch.uint8, device=DEV)
    amp = torch.ones((H, D), device=DEV)
    amp.scatter_(1, torch.rand((H, D), device=DEV, generator=gen).topk(4, dim=1).indices, 10.0)
    step = max(1, (1 << 25) // (H * page * D))
    off = _offsets(k, v)[0][torch.arange(page, device=DEV) % 16]
    for p0 in range(0, n_pages, step):
        n = min(step, n_pages - p0)
        kv = torch.randn((2, n * page, H, D), device=DEV, generator=gen)
        kv = (kv * amp).half()
        val = torch.cat(_k_bytes(kv[0], k) + _v_bytes(kv[1], v), -1)
        val = val.view(n, page // 16, 16, H, -1).permute(0, 3, 1, 2, 4).reshape(n, H, page // 16, -1)
        o = off.view(page // 16, -1).expand(n, H, page // 16, -1)
        pool[p0:p0 + n].scatter_(-1, o, val)
    return pool


# ---------------------------------------------------------------- prepare --
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7fffffff)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _buf(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    return {"qkv": _prepare_qkv, "move": _prepare_move, "fork": _prepare_fork, "copy": _prepare_copy}[case["op"]](case, g, st)


def _prepare_qkv(case, g, st):
    T, Hq, H, page = case["tokens"], case["q_heads"], case["kv_heads"], case["page"]
    lens, new = _step(case)
    ends = np.cumsum(new)
    st["lens"], st["q_start"] = _i32(lens), _i32([0] + [int(x) for x in ends])
    at = np.concatenate([np.arange(n) + L - n for L, n in zip(lens, new)])
    st["positions"] = _buf(T) if case["derived"] else _i32(at.tolist())
    if case["fused"]:   # columns of one projection's output
        x = torch.randn((T, Hq + 2 * H, D), device=DEV, generator=g).half()
        st["q16"], st["k16"], st["v16"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        st["q16"] = torch.randn((T, Hq, D), device=DEV, generator=g).half()
        st["k16"], st["v16"] = (torch.randn((T, H, D), device=DEV, generator=g).half() for _ in range(2))
    st["q_norm"], st["k_norm"] = (1 + 0.2 * torch.randn(D, device=DEV, generator=g) for _ in range(2))
    st["q_out"] = _buf(T, Hq, D, dtype=torch.float16)
    st["k_out"], st["v_out"] = (_buf(T, H, D, dtype=torch.float16) for _ in range(2))
    if case["to"] == "pages":
        blocks = [(L + page - 1) // page - (L - n) // page for L, n in zip(lens, new)]   # pages that the new tokens touch
        n_pages = sum(blocks) + 3
        ids = torch.randperm(n_pages, device=DEV, generator=g).cpu().numpy()
        slots, first = [], 0
        for L, n, m in zip(lens, new, blocks):
            pos = np.arange(L - n, L)
            slots.append(ids[first + pos // page - (L - n) // page] * page + pos % page)
            first += m
        st["slots"] = _i32(np.concatenate(slots).tolist())
        st["pool"] = torch.randint(0, 128, (n_pages, H, page // 16, _tile_bytes(case["k"], case["v"])), dtype=torch.uint8, device=DEV, generator=g)
    f, factor = _frequencies(case)
    st["freqs"], st["factor"] = torch.tensor(f, dtype=torch.float64, device=DEV), factor
    return st


def _places(case):
    """(from, to) positions of a move case's tokens in one long row of pages, and the row's length."""
    r = random.Random(case["lens_seed"])
    T = case["tokens"]
    if case["kind"] == "turn":
        return np.arange(T), np.arange(T), T
    if case["kind"] == "shift":   # the first 4 tokens stay, the next `gap` go
        to = np.arange(T) + 4
        return to + case["gap"], to, T + 4 + case["gap"]
    frm, to, at = [], [], 0       # trees of 16 tokens behind some history, up to 4 of them accepted
    while len(frm) < T:
        at += r.randint(1, 40)
        kept = sorted(r.sample(range(16), min(4, T - len(frm))))
        frm += [at + x for x in kept]
        to += [at + x for x in range(len(kept))]
        at += 16
    return np.array(frm), np.array(to), at


def _prepare_move(case, g, st):
    page, H = case["page"], case["kv_heads"]
    frm, to, L = _places(case)
    blocks = (L + page - 1) // page
    st["pool"] = _fill_pool(g, blocks + 3, H, page, case["k"], case["v"])
    ids = torch.randperm(blocks + 3, device=DEV, generator=g)
    for name, pos in (("from", frm), ("to", to)):
        pos = torch.tensor(pos, device=DEV)
        st[name] = (ids[pos // page] * page + pos % page).int()
    st["turn"] = torch.full_like(st["to"], -case["gap"])
    st["k_out"], st["v_out"] = (_buf(case["tokens"], H, D, dtype=torch.float16) for _ in range(2))
    st["freqs"] = torch.tensor(_frequencies(case)[0], dtype=torch.float64, device=DEV)
    return st


def _requests(case):
    """Lengths, the blocks that each group's members share, parents and kept positions of a fork case."""
    r = random.Random(case["lens_seed"])
    B, G = case["n_seqs"], case["group"]
    lens, shared, parent, keep = [], [], [], []
    for g in range(B // G):
        prompt = r.randint(0, case["len_hi"])
        tail = r.randint(0, max(1, (case["len_hi"] - prompt) // 4))
        ended = r.random() < case["end"]
        for i in range(G):
            b = g * G + i
            lens.append(min(case["len_hi"], prompt + tail))
            shared.append(min(prompt, lens[-1]) // case["page"])
            x = r.random()
            parent.append(-1 if ended else g * G + r.randrange(G) if r.random() < case["swap"] else b)
            keep.append(1 << 30 if x >= case["cut"] else max(0, lens[-1] - r.randint(1, 40)))
            if not ended and x < case["cut"] / 4 and b > 0:   # a new request on another's prefix
                parent[-1] = r.randrange(b)
                keep[-1] = r.randint(0, lens[parent[-1]])
    return lens, shared, parent, keep


def _prepare_fork(case, g, st):
    lens, shared, parent, keep = _requests(case)
    B, G, P = case["n_seqs"], case["group"], case["page"]
    most = (case["len_hi"] + P - 1) // P + 1
    blocks = [(n + P - 1) // P for n in lens]
    used = sum(n if b % G == 0 else n - s for b, (n, s) in enumerate(zip(blocks, shared)))
    n_pages = used + B + 7
    ids = torch.randperm(n_pages, device=DEV, generator=g).cpu().numpy()
    table = np.full((B, most), -1, np.int32)
    at = 0
    for b, (n, s) in enumerate(zip(blocks, shared)):
        s = s if b % G else 0
        table[b, :s] = table[b - b % G, :s]
        table[b, s:n] = ids[at:at + n - s]
        at += n - s
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - at] = ids[at:]
    st.update(n_pages=n_pages, lens=_i32(lens), parent=_i32(parent), keep=_i32(keep), table=torch.from_numpy(table).to(DEV),
              free=torch.from_numpy(free).to(DEV), n_free=_i32([n_pages - at]), table_out=torch.full((B, most), -1, dtype=torch.int32, device=DEV),
              lens_out=_buf(B), n_free_out=_buf(1), copy_from=_buf(B), copy_to=_buf(B), copy_held=_buf(B), status=_buf(B))
    return st


def _copies(case):
    """Positions copied of each of a copy case's pairs; 0: the pair names no pages."""
    r = random.Random(case["lens_seed"])
    held = [r.randint(1, case["page"]) if case["held"] else case["page"] for _ in range(case["n_copies"])]
    return [h if r.random() < case["share"] or case["share"] == 1.0 else 0 for h in held]


def _prepare_copy(case, g, st):
    held, n = _copies(case), case["n_copies"]
    n_pages = 2 * n + 3
    there = torch.tensor(held, device=DEV) > 0
    ids = torch.randperm(n_pages - 1, device=DEV, generator=g).int()
    st["from"] = torch.where(there, ids[:n], torch.full_like(ids[:n], -1))
    st["to"] = torch.where(there, ids[n:2 * n], torch.full_like(ids[:n], -1))
    st["held"] = _i32(held) if case["held"] else None
    st["pools"] = torch.randint(0, 256, (case["pools"], n_pages, case["kv_heads"], case["page"] // 16, _tile_bytes(case["k"], case["v"])),
                                dtype=torch.uint8, device=DEV, generator=g)
    return st


# -------------------------------------------------------------------- run --
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"qkv": _plain_qkv, "move": _plain_move, "fork": _plain_fork, "copy": _plain_copy}[op](state)


def _own_rope(kvq, case):
    if case["n_rot"] == 0:
        return None
    kind = {"none": kvq.ROPE_PLAIN, "linear": kvq.ROPE_LINEAR, "base": kvq.ROPE_BASE, "index": kvq.ROPE_BY_INDEX, "turns": kvq.ROPE_BY_TURNS}[case.get("scaling", "none")]
    fast, slow = {"index": (32.0, 1.0), "turns": (4.0, 1.0)}.get(case.get("scaling"), (0.0, 0.0))
    return kvq.Rope(case["n_rot"], 10000.0, kvq.ROPE_PAIRS if case["layout"] == "pairs" else kvq.ROPE_HALF, scaling=kind,
                    factor=8.0, original=4096.0, fast=fast, slow=slow, device=DEV)


def _own(state, op):
    """The calls a serving loop makes; the prepared calls are kept as it keeps them."""
    from quantized_kv_cache_03_gb300 import kvq
    call = state.get("call")
    if call is None:
        call = state["call"] = _own_calls(kvq, state, op)
    for c in call:
        c()
    if op == "qkv":
        if state["case"]["to"] == "plain":
            return {"q": state["q_out"], "k": state["k_out"]}
        return {"q": state["q_out"], "k": state["k_out"], "v": state["v_out"]}
    if op == "move":
        return {"k": state["k_out"], "v": state["v_out"]}
    if op == "fork":
        return {"table": state["table_out"], "lens": state["lens_out"], "free": state["free"], "n_free": state["n_free_out"],
                "from": state["copy_from"], "to": state["copy_to"], "held": state["copy_held"], "status": state["status"]}
    return state["pools"]


def _own_pool(kvq, case, data):
    return kvq.PagePool(data.shape[0], case["page"], case["kv_heads"], kvq.V_Q4_0 if case["v"] == "q4" else kvq.V_Q8_0,
                        k_type=kvq.K_I8 if case["k"] == "i8" else kvq.K_F16, data=data)


def _own_calls(kvq, s, op):
    case = s["case"]
    if op == "fork":
        return [kvq.PageForkCall(case["page"], s["n_pages"], s["lens"], s["table"], s["free"], s["n_free"], s["table_out"], s["lens_out"],
                                 s["n_free_out"], s["copy_from"], s["copy_to"], s["copy_held"], s["status"], parent=s["parent"], keep=s["keep"])]
    if op == "copy":
        return [kvq.PageCopyCall([_own_pool(kvq, case, data) for data in s["pools"]], s["from"], s["to"], held=s["held"])]
    if op == "move":
        pool = _own_pool(kvq, case, s["pool"])
        turned = dict(rope=_own_rope(kvq, case), turn=s["turn"]) if case["n_rot"] else {}
        return [kvq.PagedMoveCall(pool, s["from"], s["to"], staged=case["kind"] != "turn", **turned),
                kvq.PagedGatherCall(pool, s["to"], s["k_out"], s["v_out"])]
    calls = [kvq.PagePositionsCall(s["q_start"], s["lens"], s["positions"])] if case["derived"] else []
    rope = _own_rope(kvq, case)
    norms = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS) if case["norm"] else {}
    if case["to"] == "plain":
        return calls + [kvq.QkvCall(s["q16"], s["k16"], None, s["positions"], rope, s["q_out"], k_out=s["k_out"], **norms)]
    pool = _own_pool(kvq, case, s["pool"])
    return calls + [kvq.QkvCall(s["q16"], s["k16"], s["v16"], s["positions"], rope, s["q_out"], pool=pool, slots=s["slots"], **norms),
                    kvq.PagedGatherCall(pool, s["slots"], s["k_out"], s["v_out"])]


def _plain_norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_rotate(x, angle, factor, case):
    """x [tokens, heads, 128] in fp32 turned by angle [tokens, pairs] (float64)."""
    n = case["n_rot"]
    if n == 0:
        return x
    c, s = ((f(angle) * factor).float()[:, None, :] for f in (torch.cos, torch.sin))
    a, b = (x[..., :n // 2], x[..., n // 2:n]) if case["layout"] == "half" else (x[..., 0:n:2], x[..., 1:n:2])
    y = (a * c - b * s, a * s + b * c)
    return torch.cat(list(y) + [x[..., n:]], -1) if case["layout"] == "half" else torch.cat([torch.stack(y, -1).flatten(-2), x[..., n:]], -1)


def _plain_qkv(s):
    case = s["case"]
    pos = s["positions"].long()
    if case["derived"]:
        t = torch.arange(case["tokens"], device=DEV)
        qs = s["q_start"].long()
        b = torch.searchsorted(qs[1:], t, right=True)
        pos = s["lens"].long()[b] - qs[1:][b] + t
    angle = pos.double()[:, None] * s["freqs"]
    q, k = s["q16"].float(), s["k16"].float()
    if case["norm"]:
        q, k = _plain_norm(q, s["q_norm"]), _plain_norm(k, s["k_norm"])
    q, k = (_plain_rotate(x, angle, s["factor"], case).half() for x in (q, k))
    if case["to"] == "plain":
        return {"q": q, "k": k}
    at = _addresses(s["pool"], s["slots"].long(), case)
    s["pool"].view(-1)[at.reshape(-1)] = torch.cat(_k_bytes(k, case["k"]) + _v_bytes(s["v16"], case["v"]), -1).reshape(-1)
    kk, vv = _read_values(s["pool"].view(-1)[at], case)
    return {"q": q, "k": kk.half(), "v": vv.half()}


def _plain_move(s):
    case, turn = s["case"], s["turn"]
    flat = s["pool"].view(-1)
    b = flat[_addresses(s["pool"], s["from"].long(), case)]
    if case["n_rot"]:
        n = _offsets(case["k"], case["v"])[1]
        k = _plain_rotate(_read_values(b, case)[0], turn.double()[:, None] * s["freqs"], 1.0, case).half()
        kb = torch.cat(_k_bytes(k, case["k"]), -1)
        if case["k"] == "i8":   # blocks without a rotated value stay as they are
            still = torch.arange(NB, device=DEV) * 32 >= case["n_rot"]
            still = torch.cat([still.repeat_interleave(32), still.repeat_interleave(2)])
            kb = torch.where(still | (turn == 0)[:, None, None], b[..., :n], kb)
        b = torch.cat([kb, b[..., n:]], -1)
    flat[_addresses(s["pool"], s["to"].long(), case).reshape(-1)] = b.reshape(-1)
    k, v = _read_values(b, case)
    return {"k": k.half(), "v": v.half()}


def _plain_fork(s):
    case = s["case"]
    P, B, n_pages, bt = case["page"], case["n_seqs"], s["n_pages"], s["table"].long()
    lens, par, n_free = s["lens"].long(), s["parent"].long(), s["n_free"].long()
    some = (par >= 0) & (par < B)
    par = par.clamp(0, B - 1)
    keep = torch.where(some, torch.minimum(s["keep"].long(), lens[par]), torch.zeros_like(par)).clamp(min=0)
    rows, cols, b = bt[par], torch.arange(bt.shape[1], device=DEV)[None, :], torch.arange(B, device=DEV)

    def listed_by(t, used):   # whether each page is; one more place takes what lists none
        at = torch.where(used & (t >= 0) & (t < n_pages), t, torch.full_like(t, n_pages))
        return torch.zeros(n_pages + 1, dtype=torch.bool, device=DEV).scatter_(0, at.reshape(-1), True)[:n_pages]

    whole = keep // P
    old, full = listed_by(bt, cols < ((lens + P - 1) // P)[:, None]), listed_by(rows, cols < whole[:, None])
    tail = rows.gather(1, whole.clamp(max=bt.shape[1] - 1)[:, None]).squeeze(1)
    has = (keep % P != 0) & (tail >= 0) & (tail < n_pages)
    tail = torch.where(has, tail, torch.full_like(tail, n_pages))
    first = torch.full((n_pages + 1,), B, device=DEV).scatter_reduce_(0, tail, b, "amin")
    need = has & (torch.cat([full, full[:1]])[tail] | (first[tail] != b))
    gone = old & ~full & (first[:n_pages] == B)
    at = n_free + gone.long().cumsum(0) - 1
    at = torch.where(gone & (at < n_pages), at, torch.full_like(at, n_pages))
    stack = torch.cat([s["free"], s["free"][:1]]).scatter_(0, at, torch.arange(n_pages, device=DEV, dtype=torch.int32))[:n_pages]
    avail = (n_free + gone.sum()).clamp(max=n_pages)
    rank = need.long().cumsum(0) - need.long()
    given = need & (rank < avail)
    page = torch.where(given, stack[(avail - 1 - rank).clamp(0, n_pages - 1)].long(), torch.full_like(rank, -1))
    lens_out = torch.where(need & ~given, whole * P, keep)
    table = torch.where(cols < ((lens_out + P - 1) // P)[:, None], rows, s["table_out"].long())
    table = torch.where(given[:, None] & (cols == whole[:, None]), page[:, None], table)
    none = torch.full_like(page, -1)
    return {"table": table.int(), "lens": lens_out.int(), "free": stack, "n_free": (avail - given.sum()).int().reshape(1),
            "from": torch.where(given, tail, none).int(), "to": page.int(), "held": torch.where(given, keep % P, torch.zeros_like(keep)).int(),
            "status": (need & ~given).int()}


def _plain_copy(s):
    """Bytes of the listed pages' first tiles, page after page of every pool."""
    case, pools = s["case"], s["pools"]
    frm, to = s["from"].long(), s["to"].long()
    some = frm >= 0
    src, dst = frm.clamp(min=0), torch.where(some, to, torch.zeros_like(to))
    there = some[:, None]
    if s["held"] is not None:
        there = there & (torch.arange(case["page"] // 16, device=DEV)[None, :] < ((s["held"].long() + 15) // 16)[:, None])
    there = there.expand(-1, case["page"] // 16)[None, :, None, :, None]
    dst = torch.where(some, dst, src.new_tensor(pools.shape[1] - 1))   # pairs without pages rewrite the last page, which no pair names, as it is
    val = torch.where(there, pools[:, src], pools[:, dst])
    pools.index_copy_(1, dst, val)
    return pools


# ------------------------------------------------------------------- work --
def _row_bytes(case):
    return _tile_bytes(case["k"], case["v"]) / 16 * case["kv_heads"]


def work(case):
    op = case["op"]
    if op == "fork":
        lens, shared, parent, keep = _requests(case)
        P, B = case["page"], len(lens)
        kept = [min(n, lens[p]) if p >= 0 else 0 for n, p in zip(keep, parent)]
        entries = sum((n + P - 1) // P for n in lens), sum((n + P - 1) // P for n in kept)
        return {"bytes": 4.0 * (sum(entries) + 3 * B + 5 * B + 2), "flops": 0.0}
    if op == "copy":
        tiles = sum((h + 15) // 16 for h in _copies(case))
        return {"bytes": case["n_copies"] * 8.0 + 2.0 * tiles * case["pools"] * case["kv_heads"] * _tile_bytes(case["k"], case["v"]), "flops": 0.0}
    T, H = case["tokens"], case["kv_heads"]
    vals = T * H * D * 2.0      # K and V
    if op == "move":            # bytes in and out, the values read back
        k_row = (128 + 8 if case["k"] == "i8" else 256) * H
        moved = k_row if case["kind"] == "turn" else _row_bytes(case)
        return {"bytes": T * (2 * moved + _row_bytes(case) + 16) + vals * 2, "flops": T * H * (3.0 * case["n_rot"] + 2 * D)}
    q = T * case["q_heads"] * D
    flops = (q + vals / 2) * (3 + (4 if case["norm"] else 0)) + vals
    if case["to"] == "plain":
        return {"bytes": 2 * (2 * q + vals) + 4 * T, "flops": flops}
    return {"bytes": 2 * (2 * q + vals) + T * (2 * _row_bytes(case) + 12) + vals * 2, "flops": flops}


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


def _round_blocks(x, top, low, high):
    """One 32-block rule in 64 bits with its fp16 scale: the value each element stands for."""
    y = x.double().reshape(x.shape[:-1] + (NB, 32))
    s = (y.abs().amax(-1, keepdim=True) / top).half().double()
    r = y / torch.where(s == 0, torch.ones_like(s), s)
    c = torch.where(r < 0, torch.ceil(r - 0.5), torch.floor(r + 0.5)).clamp(low, high)
    return torch.where(s == 0, torch.zeros_like(c), c * s).reshape(x.shape)


def _turned(x, pos, case, scaling_factor):
    """x [tokens, heads, 128] turned pair by pair as complex numbers, in 64 bits."""
    n = case["n_rot"]
    if n == 0:
        return x
    f = torch.tensor(_frequencies(case)[0], dtype=torch.float64, device=x.device)
    phase = torch.remainder(pos.double()[:, None] * f, 2 * math.pi)
    z = torch.polar(torch.full_like(phase, scaling_factor), phase)[:, None, :]
    first = torch.arange(n // 2, device=x.device) * (1 if case["layout"] == "half" else 2)
    second = first + (n // 2 if case["layout"] == "half" else 1)
    w = torch.complex(x[..., first], x[..., second]) * z
    y = x.clone()
    y[..., first], y[..., second] = w.real, w.imag
    return y


def exact(case, seed):
    if case["op"] in ("fork", "copy"):
        return None
    s = prepare(case, seed)
    if case["op"] == "move":
        P, H, pool = case["page"], case["kv_heads"], s["pool"]
        frm = s["from"].long()
        K, V = _tile_values(pool.view(-1, pool.shape[-1]), case["k"], case["v"])
        K, V = (x.view(pool.shape[0], H, P, D)[frm // P, :, frm % P] for x in (K, V))
        if case["n_rot"]:
            T = _turned(K, s["turn"], case, 1.0).half().double()
            if case["k"] == "i8":
                n = (case["n_rot"] + 31) // 32 * 32
                T = torch.cat([_round_blocks(T, 127.0, -127, 127)[..., :n], K[..., n:]], -1)
            K = T
        return {"k": K, "v": V}
    lens, new = _step(case)
    pos = torch.tensor(np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)]), device=DEV)
    q, k, v = (s[n].double() for n in ("q16", "k16", "v16"))
    if case["norm"]:
        q, k = (x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / D + EPS) * s[w].double() for x, w in ((q, "q_norm"), (k, "k_norm")))
    q, k = (_turned(x, pos, case, _frequencies(case)[1]) for x in (q, k))
    if case["to"] == "plain":
        return {"q": q, "k": k}
    k = k.half().double()
    return {"q": q, "k": k if case["k"] == "f16" else _round_blocks(k, 127.0, -127, 127),
            "v": _round_blocks(v, 127.0, -127, 127) if case["v"] == "q8" else _round_blocks(v, 8.0, -8, 7)}
