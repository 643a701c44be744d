"""Shared helpers of the paged cache's GPU tests: a batch of sequences held in
pages, and what each operator has to give, from the fp64 oracle and numpy."""
import numpy as np
import torch

import oracle
from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, dev, lane_view_index

POISON = 0xFF   # as fp16 scales: NaN


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev())


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev())


def scale_index():
    """Byte offset of (position u, block b) in a scale area, read the way a
    warp does: lane c's 16 bytes of an 8-position group hold, block after
    block, the scales of positions 2c and 2c + 1."""
    idx = np.zeros((16, 4), np.int64)
    for sub in range(2):
        for c in range(4):
            for b in range(4):
                for e in range(2):
                    idx[8 * sub + 2 * c + e, b] = (sub * 4 + c) * 16 + b * 4 + 2 * e
    return idx


def split_tiles(tiles, k_type, v_type):
    """uint8 [..., tile bytes] -> dict of logical arrays [..., 16, row] as the
    oracle's quantize_kv lays a row out."""
    lead = tiles.shape[:-1]
    t = tiles.reshape(-1, tiles.shape[-1])
    n, at, out = len(t), 0, {}

    def codes(name, size, row, dtype, bias):
        nonlocal at
        idx = lane_view_index(name, v_type)
        a = np.ascontiguousarray(t[:, at:at + size]).view(dtype)
        got = np.empty((n, 16, row), dtype)
        got[:, idx[:, 1], idx[:, 2]] = a[:, idx[:, 0]]
        at += size
        return (got ^ bias).reshape(lead + (16, row)) if bias else got.reshape(lead + (16, row))

    def scales():
        nonlocal at
        a = np.ascontiguousarray(t[:, at:at + 128])
        at += 128
        si = scale_index()
        return (a[:, si].astype(np.uint16) | a[:, si + 1].astype(np.uint16) << 8).reshape(lead + (16, 4))

    if k_type == kvq.K_F16:
        out["k16"] = codes("k16", 4096, 128, np.uint16, 0)
    else:
        out["kq"] = codes("kq", 2048, 128, np.uint8, 0x80)
        out["ks"] = scales()
    q4 = v_type == kvq.V_Q4_0
    out["vq"] = codes("vq", 1024 if q4 else 2048, 64 if q4 else 128, np.uint8, 0 if q4 else 0x80)
    out["vs"] = scales()
    assert at == t.shape[1]
    return out


def pool_rows(pool):
    """Logical arrays [n_pages][H][page tokens][row] of a whole pool."""
    raw = pool.data.cpu().numpy().reshape(pool.n_pages, pool.n_kv_heads, pool.page_tokens // 16, -1)
    return {k: v.reshape(v.shape[:2] + (pool.page_tokens, v.shape[-1])) for k, v in
            split_tiles(raw, pool.k_type, pool.v_type).items()}


def f16(bits):
    return np.ascontiguousarray(bits).view(np.float16).astype(np.float64)


def values(rows, v_type):
    """fp64 K and V [..., 128] of logical rows."""
    def scaled(c, s):
        return (c.reshape(c.shape[:-1] + (4, 32)) * f16(s)[..., None]).reshape(c.shape)
    k = f16(rows["k16"]) if "k16" in rows else scaled(rows["kq"].view(np.int8).astype(np.float64), rows["ks"])
    vq = rows["vq"]
    if v_type == kvq.V_Q4_0:
        c = vq.reshape(vq.shape[:-1] + (4, 16))
        c = np.concatenate([c & 15, c >> 4], -1).astype(np.float64).reshape(vq.shape[:-1] + (128,)) - 8
    else:
        c = vq.view(np.int8).astype(np.float64)
    return k, scaled(c, rows["vs"])


def tables_ref(page, n_pages, lens, n_new, free, n_free, table, max_blocks, n_tokens):
    """kvq_page_tables in plain Python, one sequence after another."""
    lens = [min(max(int(x), 0), max_blocks * page) for x in lens]
    stack = [int(x) for x in free[:min(max(n_free, 0), n_pages)]]
    table, B = table.copy(), len(lens)
    free = free.copy()
    n_in = len(stack)

    def blocks(n):
        return -(-n // page)

    for b in range(B):
        if n_new[b] < 0:
            stack += [int(x) for x in table[b, :blocks(lens[b])]]
    stack = stack[:n_pages]
    q_start, status, lens_out = [0], [], []
    slots = np.full(n_tokens, -1, np.int32)
    out_of_pages = False
    for b in range(B):
        add = max(int(n_new[b]), 0)
        t0 = q_start[-1]
        q_start.append(t0 + add)
        st = 0
        if add:
            need = blocks(lens[b] + add) - blocks(lens[b])
            if lens[b] + add > max_blocks * page or t0 + add > n_tokens:
                st = 2
            elif need and (out_of_pages or need > len(stack)):
                st, out_of_pages = 1, True
            else:
                for j in range(need):
                    table[b, blocks(lens[b]) + j] = stack.pop()
                for i in range(add):
                    pos = lens[b] + i
                    pg = table[b, pos // page]
                    if 0 <= pg < n_pages:
                        slots[t0 + i] = pg * page + pos % page
        status.append(st)
        lens_out.append(0 if n_new[b] < 0 else lens[b] + (add if st == 0 else 0))
    for v in range(n_in, len(stack)):
        free[v] = stack[v]
    return dict(block_table=table, free=free, n_free=np.array([len(stack)]), lens=np.array(lens_out),
                q_start=np.minimum(q_start, 2 ** 31 - 1), slots=slots, status=np.array(status))


class Batch:
    """Sequences of lens[b] positions, the newest new[b] of them this step's
    rows, appended through slots into a pool whose other bytes are poison."""

    def __init__(self, lens, new, H=2, Hq=4, page=16, k_type=kvq.K_I8, v_type=kvq.V_Q4_0, seed=0, spare=3,
                 pad_rows=0, table_pad=0, outliers=False, hide=(), shape=None):
        r = np.random.default_rng(seed)
        self.lens, self.new, self.H, self.Hq, self.page = list(lens), list(new), H, Hq, page
        self.k_type, self.v_type = k_type, v_type
        B = len(lens)
        blocks = [-(-n // page) for n in lens]
        n_pages = sum(blocks) + spare
        self.pool = kvq.PagePool(n_pages, page, H, v_type, k_type=k_type)
        self.pool.data.fill_(POISON)
        ids = r.permutation(n_pages)
        self.most = max([1] + blocks)
        table = np.full((B, self.most + table_pad), -7, np.int32)
        at = 0
        for b, n in enumerate(blocks):
            table[b, :n] = ids[at:at + n]
            at += n
        self.kv = []
        for n in lens:
            kv = r.standard_normal((2, n, H, 128)).astype(np.float32)
            if outliers and n:
                kv[:, :, :, r.choice(128, 4, replace=False)] *= 10
            self.kv.append((kv if shape is None else shape(kv)).astype(np.float16))
        if sum(lens):
            slots = np.concatenate([table[b, np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(lens)])
            k16, v16 = (np.concatenate([kv[i] for kv in self.kv]) for i in range(2))
            kvq.kvq_paged_append(self.pool, to_dev(k16), to_dev(v16), i32(slots))
        for b, j in hide:   # pages taken away from a sequence: their positions are masked
            table[b, j] = -1 if (b + j) % 2 else n_pages
        self.table, self.hide = table, set(hide)
        self.T = sum(new) + pad_rows
        self.q = r.standard_normal((max(1, self.T), Hq, 128)).astype(np.float16)[:self.T]
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.max_q = max([1] + list(new))

    def attn(self, causal=True, out=torch.float32, head_map=None, scale=SM_SCALE, lse=True, q=None, stream=None,
             max_q=None, workspace=None):
        o = torch.full((self.T, self.Hq, 128), 777.0, dtype=out, device=dev())
        ls = torch.full((self.T, self.Hq), 777.0, dtype=torch.float32, device=dev()) if lse else None
        table = to_dev(self.table)[:, :self.most]
        kvq.kvq_paged_attn(self.pool, to_dev(self.q) if q is None else q, i32(self.q_start), max_q or self.max_q,
                           i32(self.lens), table, causal, scale, o, ls, head_map=head_map, stream=stream,
                           workspace=workspace)
        torch.cuda.synchronize()
        return o.float().cpu().numpy().astype(np.float64), ls.cpu().numpy().astype(np.float64) if lse else None

    def reference(self, b, causal, head_map=None, scale=SM_SCALE):
        """fp64 out and lse of sequence b's rows."""
        n, L = self.new[b], self.lens[b]
        hm = oracle.default_head_map(self.Hq, self.H) if head_map is None else np.asarray(head_map, np.int32)
        q = self.q[self.q_start[b]:self.q_start[b] + n]
        if L == 0 or n == 0:
            return np.zeros((n, self.Hq, 128)), np.full((n, self.Hq), -np.inf)
        cache = oracle.quantize_kv(*self.kv[b], self.v_type, k_type=self.k_type)
        hidden = [j for (c, j) in self.hide if c == b]
        if not hidden and L >= n:
            r = oracle.decode_seq(cache, q, hm, causal, scale, self.v_type, n_threads=8)
            return r["out"], r["lse"]
        k, v = values(cache, self.v_type)   # [H][L][128]
        qv = q.astype(np.float64)
        if self.k_type == kvq.K_I8:
            qc = oracle.quantize_kv(q, q, kvq.V_Q8_0)
            qv = values(qc, kvq.V_Q8_0)[0].transpose(1, 0, 2)
        seen = np.ones(L, bool)
        for j in hidden:
            seen[j * self.page:(j + 1) * self.page] = False
        out, lse = np.zeros((n, self.Hq, 128)), np.full((n, self.Hq), -np.inf)
        for i in range(n):
            ok = seen & (np.arange(L) <= (L - n + i if causal else L - 1))
            if not ok.any():
                continue
            for h in range(self.Hq):
                s = k[hm[h]][ok] @ qv[i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                lse[i, h] = m + np.log(p.sum())
                out[i, h] = p @ v[hm[h]][ok] / p.sum()
        return out, lse

    def bounds(self, scale=SM_SCALE, out=torch.float32):
        """How far out (absolute, and relative to the value) and lse may be off.
        A score is a sum of fp32 products of |q||k| at most (Cauchy-Schwarz):
        up to 32 roundings of 2^-24 each; a weight is off by that (natural
        units) and 2^-20 for ex2, lg2, the reciprocal and the sums; fp32 P.V
        keeps p*d to 2^-21 and rounds its running sum, about sqrt(L) * 2^-23 of
        it; fp16 output rounds p*d (2^-11) and the result (2^-11)."""
        kn = max([1e-9] + [float(np.linalg.norm(kv[0].astype(np.float64), axis=-1).max()) for kv in self.kv if kv.size])
        qn = float(np.linalg.norm(self.q.astype(np.float64), axis=-1).max()) if self.T else 0.0
        vmax = max([1e-9] + [float(np.abs(kv[1].astype(np.float64)).max()) for kv in self.kv if kv.size]) * 1.01
        es = 32 * 2.0 ** -24 * kn * qn * abs(scale) * 1.03 + 2.0 ** -20
        tail = (2.0 ** -21 + np.sqrt(max([1] + self.lens)) * 2.0 ** -23)
        a, rel = vmax * (2 * es + tail), 0.0
        if out == torch.float16:
            a, rel = a + vmax * 2.0 ** -11, 2.0 ** -11
        return a, rel, es + 2.0 ** -22 * (kn * qn * abs(scale) + 20)

    def check(self, causal=True, out=torch.float32, head_map=None, scale=SM_SCALE, what="", **kw):
        o, ls = self.attn(causal, out, head_map, scale, **kw)
        a, rel, el = self.bounds(scale, out)
        assert kvq.kvq_wait_timeouts() == 0
        for b in range(len(self.lens)):
            t0, n = self.q_start[b], self.new[b]
            ro, rl = self.reference(b, causal, head_map, scale)
            go, gl = o[t0:t0 + n], ls[t0:t0 + n]
            assert np.array_equal(np.isneginf(gl), np.isneginf(rl)), "%s seq %d: empty rows differ" % (what, b)
            fin = np.isfinite(rl)
            d = np.abs(go - ro)
            assert (d <= a + rel * np.abs(ro)).all(), "%s seq %d (L %d, n %d): out off by %.3g, allowed %.3g" % (
                what, b, self.lens[b], n, np.nanmax(d) if not np.isnan(d).any() else np.nan, a)
            dl = np.abs(gl[fin] - rl[fin])
            assert (dl <= el).all(), "%s seq %d: lse off by %.3g, allowed %.3g" % (what, b, dl.max(), el)
        rest = self.q_start[-1]
        assert (o[rest:] == 777).all() and (ls[rest:] == 777).all(), "rows behind the last sequence were touched"
        return o, ls
