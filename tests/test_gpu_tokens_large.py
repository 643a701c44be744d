"""Launches of the calls around the paged cache that are large enough for their
long loops: a warp that goes over several heads, blocks of all heads in more than
one wave, a thread that pushes more than one word of marks.  Against the same
work in small calls, bit for bit, or plain Python.  And two calls side by side."""
import numpy as np
import pytest
import torch

from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import dev
from paged_cases import i32, to_dev
from tokens_cases import fork_ref, fp16_bound, normalized, rates, rotated

pytestmark = pytest.mark.gpu

I8, F16 = kvq.K_I8, kvq.K_F16
Q4, Q8 = kvq.V_Q4_0, kvq.V_Q8_0
HALF, PAIRS = kvq.ROPE_HALF, kvq.ROPE_PAIRS
FORMATS = [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)]
# kv heads, and how many of them a warp takes: all in shares of four, a short last share, three shares, one
HEADS = [(8, 4), (7, 4), (5, 2), (3, 3)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def tokens_for(H, heads, warps):
    """Tokens from which a warp takes so many of H heads: windows of eight tokens, `warps` of them to be left for every SM."""
    sms = torch.cuda.get_device_properties(dev()).multi_processor_count
    n = 8 * -(-heads * warps * sms // H) + 3
    assert -(-n // 8) * H // (warps * sms) == heads
    return n


def held(T, page, H, k_type, v_type):
    """A pool that holds T tokens at least, of magnitudes from 2^-6 to 2^6."""
    g = torch.Generator(device=dev()).manual_seed(T)
    pool = kvq.PagePool(-(-T // page), page, H, v_type, k_type=k_type)
    T = pool.n_pages * page
    kv = torch.randn((2, T, H, 128), generator=g, device=dev()) * torch.exp2(12 * torch.rand((2, T, H, 1), generator=g, device=dev()) - 6)
    kv[0, 3, 0, 32:64] = 0
    kvq.kvq_paged_append(pool, kv[0].half(), kv[1].half(), torch.arange(T, dtype=torch.int32, device=dev()))
    return pool


def in_parts(pool, frm, to, rope=None, turn=None, part=601):
    """Moved directly by calls so small that a warp takes one head."""
    for a in range(0, len(frm), part):
        b = slice(a, a + part)
        kvq.kvq_paged_move(pool, frm[b], to[b], rope=rope, turn=None if turn is None else turn[b], staged=False)


def turns(r, n):
    """Stretches of one turn, tokens each with its own, and some that stay."""
    t = r.integers(-5000, 5000, n)
    t[n // 3:n // 2] = -517
    t[::11] = 0
    return i32(t)


# ------------------------------------------------------------------ move --
@pytest.mark.parametrize("k_type,v_type", FORMATS)
@pytest.mark.parametrize("layout,n_rot", [(HALF, 128), (PAIRS, 128), (HALF, 40), (PAIRS, 64)])
@pytest.mark.parametrize("H,heads", HEADS)
def test_keys_turned_in_place(H, heads, layout, n_rot, k_type, v_type):
    r = np.random.default_rng(H)
    n = tokens_for(H, heads, 24)
    pool = held(n + 40, 64, H, k_type, v_type)
    slots, turn, rope = i32(np.arange(n) + 5), turns(r, n), kvq.Rope(n_rot, layout=layout, device=dev())
    start = pool.data.clone()
    in_parts(pool, slots, slots, rope, turn)
    want = pool.data.clone()
    assert not torch.equal(want, start)
    pool.data.copy_(start)
    kvq.kvq_paged_move(pool, slots, slots, rope=rope, turn=turn, staged=False)
    assert torch.equal(pool.data, want)


@pytest.mark.parametrize("k_type,v_type", FORMATS)
@pytest.mark.parametrize("layout,n_rot", [(HALF, 0), (HALF, 128), (PAIRS, 40), (HALF, 64)])
@pytest.mark.parametrize("H,heads", HEADS)
def test_tokens_moved(H, heads, layout, n_rot, k_type, v_type):
    """To other pages directly; and down over themselves and in any order, staged, against two direct moves by way of other pages."""
    r = np.random.default_rng(n_rot)
    n, page = tokens_for(H, heads, 24), 32
    half = -(-(n + 9) // page) * page
    pool = held(2 * half, page, H, k_type, v_type)
    cut = pool.data.numel() // 2
    start, turn = pool.data.clone(), turns(r, n) if n_rot else None
    rope = kvq.Rope(n_rot, layout=layout, device=dev()) if n_rot else None
    there = i32(half + np.arange(n))
    mixed = r.permutation(half)[:n], r.permutation(half)[:n]
    for frm, to in ((np.arange(n) + 9, np.arange(n)), mixed):
        frm[::97], to[5::101] = -1, 2 ** 30          # tokens without a slot
        ok = i32(np.where((frm >= 0) & (to < 2 ** 30), half + np.arange(n), -1))
        frm, to = i32(frm), i32(to)
        pool.data.copy_(start)
        in_parts(pool, frm, there, rope, turn)
        away = pool.data.clone()
        in_parts(pool, ok, to)
        want = pool.data[:cut].clone()
        pool.data.copy_(start)
        kvq.kvq_paged_move(pool, frm, there, rope=rope, turn=turn, staged=False)
        assert torch.equal(pool.data, away)
        pool.data.copy_(start)
        kvq.kvq_paged_move(pool, frm, to, rope=rope, turn=turn, staged=True)
        assert torch.equal(pool.data[:cut], want) and torch.equal(pool.data[cut:], start[cut:])


# ---------------------------------------------------------------- gather --
@pytest.mark.parametrize("k_type,v_type", FORMATS)
@pytest.mark.parametrize("H,heads", HEADS)
def test_gathered(H, heads, k_type, v_type):
    """Against calls of fewer rows than the kernel for many takes."""
    r = np.random.default_rng(heads)
    n, part = tokens_for(H, heads, 48), 4095 // H
    pool = held(5000, 128, H, k_type, v_type)
    slots = r.integers(0, pool.n_pages * 128, n)
    slots[:3000] = np.arange(3000) + 1
    slots[::89], slots[7::97] = -1, 2 ** 30
    slots = i32(slots)
    for dt in (torch.float32, torch.float16):
        one, two = (torch.full((2, n, H, 128), 777.0, dtype=dt, device=dev()) for _ in range(2))
        kvq.kvq_paged_gather(pool, slots, one[0], one[1])
        for a in range(0, n, part):
            b = slice(a, a + part)
            kvq.kvq_paged_gather(pool, slots[b], two[0, b], two[1, b])
        assert torch.equal(one, two)


# ------------------------------------------------------------------- qkv --
def qkv_tokens(waves, extra):
    """Tokens of so many full waves of blocks (three to an SM, eight tokens each), and some that are shared out."""
    return 24 * waves * torch.cuda.get_device_properties(dev()).multi_processor_count + extra


@pytest.mark.parametrize("layout,n_rot,norm", [(HALF, 128, False), (PAIRS, 128, True), (HALF, 40, True), (HALF, 64, False), (PAIRS, 24, False), (HALF, 0, True)])
@pytest.mark.parametrize("to", ["rows", "in place"] + FORMATS)
@pytest.mark.parametrize("waves,extra,Hq,H", [(1, 2, 9, 3), (1, 409, 12, 2), (2, 1207, 3, 5), (1, 3001, 0, 2)])
def test_new_tokens_in_more_than_a_wave(waves, extra, Hq, H, to, layout, n_rot, norm):
    """One call, and calls of less than a wave."""
    r = np.random.default_rng(extra)
    T, page, part = qkv_tokens(waves, extra), 32, 611
    g = torch.Generator(device=dev()).manual_seed(T)
    x = torch.randn((T, Hq + 2 * H, 128), generator=g, device=dev()).half()
    n_pages = -(-T // page) + 3
    order = np.concatenate([np.arange(1, T // 2), r.permutation(np.arange(T // 2, n_pages * page))])[:T]      # neighbours, and none
    slots = i32(np.where(r.random(T) < 0.1, np.where(r.random(T) < 0.5, -1, n_pages * page + 5), order))
    pos, rope = i32(r.integers(0, 131072, T)), kvq.Rope(n_rot, layout=layout, device=dev())
    w = torch.randn((2, 128), generator=g, device=dev()) if norm else [None, None]
    got = []
    for step in (T, part):
        t = x.clone()
        qo = t[:, :Hq] if to == "in place" else torch.full((T, Hq, 128), 3.0, dtype=torch.float16, device=dev())
        if to in FORMATS:
            pool = kvq.PagePool(n_pages, page, H, to[1], k_type=to[0])
            pool.data.fill_(0)
            res = pool.data
        else:
            res = ko = t[:, Hq:Hq + H] if to == "in place" else torch.full((T, H, 128), 3.0, dtype=torch.float16, device=dev())
        for a in range(0, T, step):
            b = slice(a, a + step)
            keys = dict(v16=t[b, Hq + H:], pool=pool) if to in FORMATS else dict(v16=None, k_out=ko[b])
            kvq.kvq_qkv(t[b, :Hq] if Hq else None, t[b, Hq:Hq + H], positions=pos[b], rope=rope, q_out=qo[b] if Hq else None, slots=slots[b], q_norm=w[0], k_norm=w[1], **keys)
        got.append((qo.contiguous().view(torch.int16), res.contiguous().view(torch.int16), t[:, Hq + H:]))
    for one, two in zip(*got):
        assert torch.equal(one, two)
    assert torch.equal(got[0][2], x[:, Hq + H:])
    if to == "rows":       # and the first and last of them by the formula
        f, pick = rates(n_rot)[0], np.r_[0:40, T - 40:T]
        out = slots.cpu().numpy()[pick] < 0
        for a, b, o, wt in ((0, Hq, qo, w[0]), (Hq, Hq + H, ko, w[1])):
            y, size = rotated(normalized(x[pick, a:b].cpu().numpy(), None if wt is None else wt.cpu().numpy(), 1e-6), pos.cpu().numpy()[pick], f, 1.0, layout)
            o = o[pick].cpu().numpy().astype(np.float64)
            assert (np.abs(o - y) <= fp16_bound(y, size))[~out].all() and (o[out] == 3).all()


# ------------------------------------------------------------------ fork --
def test_fork_over_nine_million_pages():
    """Several words of four pages' marks to a thread: pages given back that fill a thread's share, cross from one share and one
    block to the next, lie in its later words alone, and the last word, of one page."""
    r = np.random.default_rng(3)
    B, page, most, n_pages = 40, 16, 2000, 9_000_001
    words = -(-n_pages // 4)
    of_block = -(-words // 1024)                                  # a block's, and a thread's
    per = -(-of_block // 1024)
    assert per > 2 and words % of_block and n_pages % 4 == 1
    runs = [np.arange(5 * 4 * per), 4 * of_block * 7 - 50 + np.arange(100), 4 * (of_block * 500 + per * 3 + 1) + np.arange(4 * (per - 1)), n_pages - 1 - np.arange(77)]
    listed = np.unique(np.concatenate(runs + [r.integers(0, n_pages, 60000)]))
    listed = r.permutation(listed)[:B * most]
    others = np.setdiff1d(r.integers(0, n_pages, 4000), listed)[:1000]
    table = np.full((B, most), -9, np.int32)
    lens = np.zeros(B, np.int64)
    for b in range(B):
        row = listed[b::B]
        table[b, :len(row)], lens[b] = row, len(row) * page - r.integers(0, page)
    free = np.full(n_pages, -5, np.int32)
    free[:len(others)] = others
    for parent, keep in ((np.where(r.random(B) < 0.3, np.arange(B), -1), None), (np.full(B, B), None), (r.integers(0, 4, B), r.integers(0, 300 * page, B))):
        ref = fork_ref(page, n_pages, lens, table, free, len(others), np.full((B, most), -8, np.int32), most, parent, keep)
        o = dict(table_out=torch.full((B, most), -8, dtype=torch.int32, device=dev()), lens=i32(np.zeros(B)), n_free=i32([0]), free=to_dev(free),
                 **{k: i32(np.full(B, 99)) for k in ("copy_from", "copy_to", "copy_held", "status")})
        kvq.kvq_page_fork(page, n_pages, i32(lens), to_dev(table), o["free"], i32([len(others)]), o["table_out"], o["lens"], o["n_free"], o["copy_from"], o["copy_to"],
                          o["copy_held"], o["status"], parent=i32(parent), keep=None if keep is None else i32(keep))
        assert ref["n_free"][0] > len(others)
        for k, v in ref.items():
            assert np.array_equal(o[k].cpu().numpy(), v), k


# ---------------------------------------------------------- two at a time --
@pytest.mark.parametrize("n", [200, 9000])
def test_two_moves_at_once(n):
    """Captured on two streams with a workspace each, replayed side by side."""
    H, rope = 8, kvq.Rope(128, device=dev())
    pools = [held(n + 40 + i, 64, H, I8, Q8) for i in range(2)]
    start = [p.data.clone() for p in pools]
    frm, to, turn = i32(np.arange(n) + 31), i32(np.arange(n)), i32(np.full(n, -31))
    want = []
    for p, s in zip(pools, start):
        kvq.kvq_paged_move(p, frm, to, rope=rope, turn=turn)
        want.append(p.data.clone())
        p.data.copy_(s)
    calls = [kvq.PagedMoveCall(p, frm, to, rope, turn) for p in pools]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    for c, g in zip(calls, graphs):
        with torch.cuda.graph(g):
            c()
    for _ in range(5):
        for p, s in zip(pools, start):
            p.data.copy_(s)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.data, w) for p, w in zip(pools, want))


@pytest.mark.parametrize("B,most,n_pages", [(300, 40, 5000), (1500, 100, 200000)])
def test_two_forks_at_once(B, most, n_pages):
    """Of each size (one cluster, the whole GPU), with a workspace each."""
    page, places = 16, []
    for seed in range(2):
        r = np.random.default_rng(seed)
        table = r.permutation(n_pages)[np.arange(B * most) % (n_pages - 50)].reshape(B, most).astype(np.int32)
        lens, parent, keep = r.integers(0, most * page + 1, B), r.integers(-1, B, B), r.integers(0, most * page, B)
        free = np.full(n_pages, -5, np.int32)
        free[:50] = np.arange(50)
        ref = fork_ref(page, n_pages, lens, table, free, 50, np.full((B, most), -8, np.int32), most, parent, keep)
        o = dict(table_out=torch.full((B, most), -8, dtype=torch.int32, device=dev()), lens=i32(np.zeros(B)), n_free=i32([0]), free=to_dev(free),
                 **{k: i32(np.full(B, 99)) for k in ("copy_from", "copy_to", "copy_held", "status")})
        call = kvq.PageForkCall(page, n_pages, i32(lens), to_dev(table), o["free"], i32([50]), o["table_out"], o["lens"], o["n_free"], o["copy_from"], o["copy_to"],
                                o["copy_held"], o["status"], parent=i32(parent), keep=i32(keep))
        places.append((call, o, ref, torch.cuda.Stream(), free))
    for _ in range(5):
        for _, o, _, _, free in places:
            o["free"].copy_(to_dev(free))
        torch.cuda.synchronize()
        for call, _, _, s, _ in places:
            call(s)
        torch.cuda.synchronize()
        for _, o, ref, _, _ in places:
            for k, v in ref.items():
                assert np.array_equal(o[k].cpu().numpy(), v), k
