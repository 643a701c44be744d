"""The paged cache on a GPU: tables, append, gather and attention against plain
fp64 / Python implementations, at the sizes, masks and layouts where each can go
wrong, and the operators in a row as a server runs them."""
import numpy as np
import pytest
import torch

import oracle
from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, Case, dev
from paged_cases import POISON, Batch, f16, i32, pool_rows, tables_ref, to_dev, values

pytestmark = pytest.mark.gpu

I8, F16 = kvq.K_I8, kvq.K_F16
Q4, Q8 = kvq.V_Q4_0, kvq.V_Q8_0


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# ---------------------------------------------------------------- tables --
def _table_state(r, B, page, most, n_pages, hi, stride_pad=0):
    lens = r.integers(0, hi + 1, B)
    blocks = -(-lens // page)
    ids = r.permutation(n_pages)
    assert blocks.sum() <= n_pages
    table = np.full((B, most + stride_pad), -9, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = ids[at:at + blocks[b]]
        at += blocks[b]
    free = np.full(n_pages, -5, np.int32)
    free[:n_pages - at] = ids[at:]
    return lens, table, free, n_pages - at


def _run_tables(page, n_pages, lens, n_new, free, n_free, table, most, n_tokens, in_place=False, slot_shift=0):
    d = dict(lens=i32(lens), n_new=i32(n_new), free=to_dev(free), n_free=i32([n_free]), table=to_dev(table))
    B = len(lens)
    out = dict(lens=d["lens"] if in_place else i32(np.full(B, 99)), n_free=d["n_free"] if in_place else i32([99]),
               q_start=i32(np.full(B + 1, 99)), status=i32(np.full(B, 99)))
    buf = i32(np.full(n_tokens + slot_shift + 1, 99))
    slots = buf[slot_shift:slot_shift + n_tokens]
    kvq.kvq_page_tables(page, n_pages, d["lens"], d["n_new"], d["free"], d["n_free"], d["table"][:, :most], out["lens"],
                        out["n_free"], out["q_start"], slots, out["status"])
    torch.cuda.synchronize()
    assert int(buf[-1]) == 99 and (buf[:slot_shift] == 99).all()
    return dict(block_table=d["table"], free=d["free"], slots=slots, **out)


def _same_tables(got, ref):
    for k, v in ref.items():
        g = got[k].cpu().numpy()
        assert np.array_equal(g, v), "%s differs at %s: %s, not %s" % (k, np.argwhere(g != v)[:4].tolist(), g[g != v][:4], np.asarray(v)[g != v][:4])


@pytest.mark.parametrize("B,page,hi,chunk,release,pages,slack", [
    (1, 16, 40, 1, 0.0, 20, 0), (7, 32, 100, 9, 0.3, 60, 3), (256, 64, 900, 1, 0.0, 4300, 0), (1000, 16, 200, 70, 0.2, 14000, 0),
    (513, 128, 3, 5, 0.1, 600, 17), (4096, 16, 30, 2, 0.2, 9000, 5), (64, 256, 4000, 700, 0.5, 1300, 0)])
def test_tables(B, page, hi, chunk, release, pages, slack):
    r = np.random.default_rng(B)
    most = -(-(hi + chunk) // page) + 1
    lens, table, free, n_free = _table_state(r, B, page, most, pages, hi, stride_pad=slack)
    n_new = np.where(r.random(B) < release, -1 - r.integers(0, 3, B), np.where(r.random(B) < 0.2, 0, r.integers(1, chunk + 1, B)))
    n_tokens = int(np.maximum(n_new, 0).sum()) + slack
    ref = tables_ref(page, pages, lens, n_new, free, n_free, table, most, n_tokens)
    assert not ref["status"].any()
    for kw in (dict(), dict(in_place=True), dict(slot_shift=1)):
        _same_tables(_run_tables(page, pages, lens, n_new, free, n_free, table, most, n_tokens, **kw), ref)


def test_tables_of_nothing():
    ref = tables_ref(16, 4, [], [], np.arange(4, dtype=np.int32), 4, np.zeros((0, 2), np.int32), 2, 3)
    _same_tables(_run_tables(16, 4, np.zeros(0, int), np.zeros(0, int), np.arange(4, dtype=np.int32), 4, np.zeros((0, 2), np.int32), 2, 3), ref)


@pytest.mark.parametrize("seed", range(6))
def test_tables_short_of_pages_rows_and_tokens(seed):
    """Requests that do not fit: too few pages, too long for a row, too many rows."""
    r = np.random.default_rng(seed)
    B, page, most, pages = 40, 16, 5, 150
    lens, table, free, n_free = _table_state(r, B, page, most, pages, 60)
    n_new = r.choice([-1, 0, 1, 3, 30, 90, 2 ** 31 - 1], B)
    n_tokens = [400, 60, 0, 2000, 1, 33][seed]
    if seed % 2:
        n_free = min(n_free, 3)
        n_new = np.maximum(n_new, 0)
    ref = tables_ref(page, pages, lens, n_new, free, n_free, table, most, n_tokens)
    assert ref["status"].any()
    _same_tables(_run_tables(page, pages, lens, n_new, free, n_free, table, most, n_tokens), ref)


@pytest.mark.parametrize("seed", range(3))
def test_tables_of_many_rows(seed):
    """More rows than one pass of the table launch fills, some of them refused."""
    r = np.random.default_rng(seed)
    B, page, most, pages = 300, 64, 40, 6000
    lens, table, free, n_free = _table_state(r, B, page, most, 6000, 1000)
    n_free = min(n_free, [6000, 1100, 6000][seed])
    n_new = r.choice([-1, 0, 1, 100, 399, 2000], B)
    n_tokens = int(np.maximum(n_new, 0).sum()) + [37, 0, -20000][seed]
    assert n_tokens > 16384
    ref = tables_ref(page, pages, lens, n_new, free, n_free, table, most, n_tokens)
    assert ref["status"].any()
    for kw in (dict(), dict(in_place=True), dict(slot_shift=1)):
        _same_tables(_run_tables(page, pages, lens, n_new, free, n_free, table, most, n_tokens, **kw), ref)


def test_tables_given_back_more_pages_than_an_int_counts():
    """33 sequences that claim 2^26 pages each end: the stack fills up with the
    first ones' and what follows is dropped."""
    B, page, most, n_pages = 33, 16, 1 << 26, 64
    table = torch.empty((B, most), dtype=torch.int32, device=dev())
    table[:, :n_pages] = torch.arange(n_pages, dtype=torch.int32, device=dev())
    free = i32(np.full(n_pages, -5))
    n_free, lens_out, q_start, slots, status = i32([3]), i32(np.full(B, 9)), i32(np.full(B + 1, 9)), i32([]), i32(np.full(B, 9))
    kvq.kvq_page_tables(page, n_pages, i32(np.full(B, 1 << 30)), i32(np.full(B, -1)), free, n_free, table, lens_out, n_free, q_start,
                        slots, status)
    torch.cuda.synchronize()
    assert free.tolist() == [-5] * 3 + list(range(n_pages - 3)) and n_free.tolist() == [n_pages]
    assert not lens_out.any() and not q_start.any() and not status.any()


def test_tables_hold_bad_values_to_their_bounds():
    """Negative and too long lengths, a stack size out of range, page entries outside the pool."""
    page, pages, most = 16, 30, 4
    table = np.array([[3, -1, 0, 0], [99, 0, 0, 0], [1, 2, 4, 5], [6, 0, 0, 0]], np.int32)
    free = np.arange(10, 40, dtype=np.int32)
    lens, n_new = np.array([20, 5, 1000, -50]), np.array([10, 4, 1, 2])
    for n_free in (-3, 30, 1000):
        ref = tables_ref(page, pages, lens, n_new, free, n_free, table, most, 20)
        got = _run_tables(page, pages, lens, n_new, free, n_free, table, most, 20)
        _same_tables(got, ref)
    assert ref["status"].tolist() == [0, 0, 2, 0] and (ref["slots"][:14] == -1).all()


# ------------------------------------------------------- append and gather --
@pytest.mark.parametrize("k_type", [I8, F16])
@pytest.mark.parametrize("v_type", [Q4, Q8])
@pytest.mark.parametrize("tokens,H,page", [(1, 1, 16), (5, 3, 32), (130, 8, 64), (257, 2, 128), (64, 1, 256)])
def test_append_and_gather(tokens, H, page, k_type, v_type):
    """Bytes of every written position, poison everywhere else; the gather's
    values are exact (code * scale fits 24 bits), fp16 ones rounded once."""
    r = np.random.default_rng(tokens + page)
    n_pages = -(-tokens // page) + 2
    kv = (r.standard_normal((2, tokens, H, 128)) * r.choice([1e-4, 1, 300], (2, tokens, H, 1))).astype(np.float16)
    kv[0, 0, 0, :32] = 0                      # an all-zero block
    kv[1, tokens // 2, H - 1, 32:64] = 0
    kv[1, 0, 0, 64] = 65504                   # the largest value
    x = torch.zeros((tokens, 3 * H, 128), dtype=torch.float16, device=dev())
    x[:, H:2 * H], x[:, 2 * H:] = to_dev(kv[0]), to_dev(kv[1])
    for order in ("runs", "scattered", "backwards"):
        if order == "scattered":
            slots = r.permutation(n_pages * page)[:tokens]
        else:
            slots = page // 2 + np.arange(tokens)
            slots = slots[::-1].copy() if order == "backwards" else slots
        pool = kvq.PagePool(n_pages, page, H, v_type, k_type=k_type)
        pool.data.fill_(POISON)
        kvq.kvq_paged_append(pool, x[:, H:2 * H], x[:, 2 * H:], i32(slots))
        rows = pool_rows(pool)
        want = oracle.quantize_kv(kv[0], kv[1], v_type, k_type=k_type)
        for name, ref in want.items():
            got = rows[name][slots // page, :, slots % page]
            assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(ref.transpose(1, 0, 2)).view(np.uint8)), (name, order)
        raw = torch.full_like(pool.data, POISON).cpu().numpy()
        other = np.ones((n_pages, page), bool)
        other[slots // page, slots % page] = False
        for name, a in rows.items():
            flip = 0x80 if name == "kq" or (name == "vq" and v_type == Q8) else 0
            assert (a.transpose(0, 2, 1, 3)[other].view(np.uint8) == (POISON ^ flip)).all(), name
        k, v = values({n: a.transpose(1, 0, 2) if a.ndim == 3 else a for n, a in want.items()}, v_type)
        again = np.concatenate([slots, slots[:3], [-1, n_pages * page, -2 ** 31]])
        for dt in (torch.float32, torch.float16):
            ko, vo = (torch.full((len(again), H, 128), 777.0, dtype=dt, device=dev()) for _ in range(2))
            kvq.kvq_paged_gather(pool, i32(again), ko, vo)
            for o, ref in ((ko, k), (vo, v)):
                ref = np.concatenate([ref, ref[:3], np.full((3, H, 128), 777.0)])
                with np.errstate(over="ignore"):
                    ref = ref.astype(np.float32 if dt == torch.float32 else np.float16)
                assert np.array_equal(o.cpu().numpy()[:-3], ref[:-3]) and (o[-3:] == 777).all()


@pytest.mark.parametrize("v_type", [Q4, Q8])
def test_append_rounds_halves_as_the_rule_says(v_type):
    """Blocks full of values at, just below and just above the halves of their
    scale, at scales from fp16's subnormals to its largest, and with
    infinities and NaN among them (whose own codes say nothing)."""
    r = np.random.default_rng(3)
    n, H = 512, 4
    top = np.exp2(r.uniform(-25, 16, (n, H, 4, 1))).clip(0, 65504).astype(np.float16)
    top[:8] = np.array([0, 2.0 ** -24, 3 * 2.0 ** -24, 190 * 2.0 ** -24, 2.0 ** -14, 65504, 1, 127], np.float16)[:, None, None, None]
    kv = []
    for most in (127, 8 if v_type == Q4 else 127):
        s = (top.astype(np.float32) / np.float32(most)).astype(np.float16).astype(np.float64)
        x = ((r.integers(0, most, (n, H, 4, 32)) + 0.5) * s).clip(0, 65504).astype(np.float16)
        x = np.abs(x).view(np.int16) + r.integers(-1, 2, x.shape).astype(np.int16)
        x = np.minimum(x.clip(0).astype(np.int16), top.view(np.int16)).view(np.float16)
        x = np.where(r.random(x.shape) < 0.5, x, -x)
        x[..., 5:6] = top * np.where(r.random(top.shape) < 0.5, 1, -1).astype(np.float16)
        x[20:23, :, 1, 7] = np.array([np.inf, -np.inf, np.nan], np.float16)[:, None]
        kv.append(np.ascontiguousarray(x.reshape(n, H, 128)))
    for first in (0, 7):   # in pairs, and at an odd place first
        pool = kvq.PagePool(9, 64, H, v_type)
        pool.data.fill_(POISON)
        slots = first + np.arange(n)
        kvq.kvq_paged_append(pool, to_dev(kv[0]), to_dev(kv[1]), i32(slots))
        rows = pool_rows(pool)
        for name, ref in oracle.quantize_kv(kv[0], kv[1], v_type).items():
            got = rows[name][slots // 64, :, slots % 64]
            ref = np.ascontiguousarray(ref.transpose(1, 0, 2))
            if name in ("kq", "vq"):
                for a in (got, ref):
                    a.view(np.uint8)[20:23, :, 32 + 7 if a.shape[2] == 128 else 16 + 7] &= 0xF0 if a.shape[2] == 64 else 0
            else:   # infinity / 127 or 8 is infinity (the oracle takes an infinity's exponent, which C leaves open)
                ref.view(np.uint16)[20:22, :, 1] = 0x7C00
            bad = np.argwhere(got.view(np.uint8) != ref.view(np.uint8))
            assert not len(bad), (name, len(bad), bad[:4], got.view(np.uint8)[tuple(bad[0])], ref.view(np.uint8)[tuple(bad[0])])


def test_append_skips_rows_without_a_slot():
    pool = kvq.PagePool(2, 16, 2, Q8)
    pool.data.fill_(POISON)
    k = torch.randn((6, 2, 128), device=dev()).half()
    kvq.kvq_paged_append(pool, k, k, i32([-1, 32, 2 ** 31 - 1, -2 ** 31, 33, 1000]))
    assert (pool.data == POISON).all()
    kvq.kvq_paged_append(pool, k, k, i32([-1, 31, -1, 0, 32, -1]))
    want = oracle.quantize_kv(k.cpu().numpy(), k.cpu().numpy(), Q8)
    rows = pool_rows(pool)
    for tok, slot in ((1, 31), (3, 0)):
        assert np.array_equal(rows["kq"][slot // 16, :, slot % 16], want["kq"][:, tok].view(np.uint8))
        assert np.array_equal(rows["vs"][slot // 16, :, slot % 16], want["vs"][:, tok])


# ------------------------------------------------------------- attention --
@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 1), (10, 2), (8, 1), (16, 1), (9, 3), (20, 1)])
def test_decode_of_a_ragged_batch(Hq, H, out, k_type, v_type):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300, 0, 1000]
    b = Batch(lens, [1] * len(lens), H=H, Hq=Hq, page=16, k_type=k_type, v_type=v_type, seed=Hq, pad_rows=2, table_pad=3)
    b.new[14] = 1     # a row of a sequence that holds nothing
    b.check(out=out)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q8)])
def test_chunks_of_a_ragged_batch(page, causal, out, k_type, v_type):
    lens = [300, 37, 64, 129, 5, 0, 511, 40, 1]
    new = [7, 37, 1, 64, 5, 0, 100, 33, 1]
    Batch(lens, new, H=2, Hq=6, page=page, k_type=k_type, v_type=v_type, seed=page, pad_rows=5, outliers=True).check(causal=causal, out=out)


@pytest.mark.parametrize("new,L", [(1, 4500), (2, 5000), (3, 2500), (4, 3333), (9, 2222), (17, 3000), (33, 2049), (64, 1111), (128, 1500),
                                   (129, 700), (255, 256), (256, 256), (257, 900), (400, 400)])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
@pytest.mark.parametrize("v_type", [Q4, Q8])
def test_one_sequence_cut_into_pieces(new, L, out, v_type):
    """Row tiles that many CTAs share, and query chunks of every size class."""
    Batch([L], [new], H=1, Hq=4, page=32, v_type=v_type, seed=new, pad_rows=1).check(out=out)


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("new,L,out,v_type", [
    (64, 32768, torch.float32, Q4), (64, 20000, torch.float32, Q8), (160, 32768, torch.float16, Q8), (512, 32768, torch.float16, Q4),
    (8, 32768, torch.float32, Q8)])
def test_long_sums(new, L, out, v_type, rising):
    """Sums over many thousand positions, values of one sign: nothing may be
    lost to the accumulators' rounding, nor where their parts are joined, with
    a maximum that stays (rising = False) or keeps rising along the sequence."""
    def shape(kv):
        kv[1] = 1 + 0.25 * kv[1]
        if rising:
            kv[0] += 4 * np.arange(L, dtype=np.float32)[:, None, None] / L
        return kv
    b = Batch([L], [new], H=8, Hq=32, page=64, v_type=v_type, seed=new, shape=shape)
    if rising:
        b.q += np.float16(1)
    o, ls = b.attn(out=out)
    rows = sorted({0, new // 2, new - 1})
    k, v = values(oracle.quantize_kv(*b.kv[0], v_type), v_type)
    q = values(oracle.quantize_kv(b.q[rows], b.q[rows], Q8), Q8)[0].transpose(1, 0, 2)
    ro, rl = np.zeros((len(rows), 32, 128)), np.zeros((len(rows), 32))
    for i, t in enumerate(rows):
        n = L - new + t + 1
        for h in range(32):
            s = k[h // 4, :n] @ q[i, h] * SM_SCALE
            p = np.exp(s - s.max())
            rl[i, h], ro[i, h] = s.max() + np.log(p.sum()), p @ v[h // 4, :n] / p.sum()
    a, rel, el = b.bounds(out=out)
    assert (np.abs(o[rows] - ro) <= a + rel * np.abs(ro)).all() and (np.abs(ls[rows] - rl) <= el).all()
    # on the average the roundings cancel, unless they lean to one side.  At most 1024 positions (fp32
    # output) or 8192 are summed in accumulators that cut off, by 2^-24 of the sum on the average, with
    # three or two additions per 16 positions.  fp16 outputs are rounded, to nearest: 2^-12 over the
    # root of some thousand values.
    lean = (192 if out == torch.float32 else 1024) * 2.0 ** -24 + (2.0 ** -20 if out == torch.float32 else 2.0 ** -15)
    assert abs((o[rows] - ro).sum() / ro.sum()) <= lean


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing_and_more_rows_than_positions(causal):
    """len < new: the first rows of a causal chunk see no position."""
    for new in (3, 40, 200):
        Batch([1, 0, 2, new - 1, new], [new] * 5, H=2, Hq=4, page=16, seed=new).check(causal=causal)


@pytest.mark.parametrize("new", [1, 5, 70])
@pytest.mark.parametrize("v_type", [Q4, Q8])
@pytest.mark.parametrize("page", [16, 64])
def test_hidden_pages(new, v_type, page):
    """Table entries outside the pool hide their positions, all of them too;
    what was never written (NaN scales here) is never seen."""
    lens = [5 * page + 3, 3 * page, page, 9 * page + 1, 2 * page - 1]
    hide = [(0, 0), (0, 3), (1, 2), (2, 0), (3, 9), (3, 0), (3, 1), (3, 4)]
    Batch(lens, [new if n >= new else 1 for n in lens], H=2, Hq=4, page=page, v_type=v_type, seed=new, hide=hide).check()


def test_head_maps():
    for hm, H in (([1, 0, 1, 1, 0], 2), ([2, 2, 2, 2, 2, 2, 2, 2, 2, 0], 3), ([0, 1, 2, 3], 4)):
        for new in (1, 6, 50):
            Batch([100, 333], [new, 1], H=H, Hq=len(hm), page=16, seed=new).check(head_map=hm)


def test_shared_pages_and_the_same_sequence_twice():
    """Two sequences over one prefix read the same pages."""
    b = Batch([200, 200], [4, 4], H=2, Hq=4, page=32, seed=3)
    b.table[1] = b.table[0]
    b.kv[1] = b.kv[0]
    b.q[4:8] = b.q[:4]
    b.check()


def test_strided_queries_missing_lse_scale_and_bound():
    b = Batch([90, 300, 17], [3, 40, 17], H=2, Hq=4, page=16, seed=8)
    wide = torch.full((b.T, 9, 128), float("nan"), dtype=torch.float16, device=dev())
    wide[:, 2:6] = to_dev(b.q)
    o, ls = b.check(q=wide[:, 2:6])
    o2, none = b.attn(lse=False)
    assert none is None and np.array_equal(o, o2)
    b.check(scale=-0.3)
    b.check(scale=0.0)
    o3, ls3 = b.attn(max_q=5)     # rows past max_q are left alone
    for s in range(3):
        t0, n = b.q_start[s], b.new[s]
        assert (o3[t0 + 5:t0 + n] == 777).all() and (ls3[t0 + 5:t0 + n] == 777).all()
    assert np.array_equal(ls3[:3] != 777, ls[:3] != 777)


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q8)])
@pytest.mark.parametrize("max_q", [2, 7, 40])
def test_fewer_rows_than_announced(max_q, k_type, v_type):
    """A batch whose n_tokens leaves room for max_q rows of every sequence is
    taken by one launch, whatever q_start then holds."""
    new = [1, max_q, 0, 1, max_q - 1]
    b = Batch([300, 129, 40, 1, 77], new, H=2, Hq=8, page=32, k_type=k_type, v_type=v_type, seed=max_q,
              pad_rows=5 * max_q - sum(new))
    one = Batch([200], [max_q - 1], H=2, Hq=8, page=16, k_type=k_type, v_type=v_type, seed=max_q, pad_rows=1)
    for out in (torch.float32, torch.float16):
        b.check(out=out)
        one.check(out=out, max_q=max_q)


@pytest.mark.parametrize("new", [2, 6, 40])
def test_a_key_that_is_not_finite_stays_with_the_rows_that_see_it(new):
    for bad in (np.inf, -np.inf, np.nan):
        def shape(kv):
            kv[0][-1, :, 7::32] = bad
            return kv
        clean, b = (Batch([200], [new], H=2, Hq=8, page=16, seed=new, shape=f) for f in (None, shape))
        o, ls = b.attn()
        ro, rl = clean.reference(0, True)
        a, rel, el = clean.bounds()
        assert (np.abs(o[:-1] - ro[:-1]) <= a + rel * np.abs(ro[:-1])).all() and (np.abs(ls[:-1] - rl[:-1]) <= el).all()


def test_tensors_of_another_device_are_refused(monkeypatch):
    b = Batch([20], [1], H=1, Hq=2, page=16)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        b.attn()


def test_bad_row_ranges_touch_nothing_else():
    """q_start past the rows, decreasing or negative: clamped, nothing behind the arrays."""
    b = Batch([50, 60, 70], [2, 2, 2], H=1, Hq=2, page=16, seed=1)
    for qs in ([0, 2, 1 << 20, 1 << 20], [-5, -1, 4, 6], [0, 4, 2, 6], [9, 9, 9, 9]):
        b.q_start = np.array(qs, np.int32)
        o, ls = b.attn()
        assert np.isfinite(o).all()


def test_lengths_past_the_table_are_held_to_it():
    b = Batch([64, 100], [1, 2], H=2, Hq=4, page=16, seed=2)
    o, ls = b.check()
    full = list(b.lens)
    b.lens = [1 << 30, 100]
    b.table = b.table[:, :7].copy()
    b.table[0, 4:] = -1
    b.most = 7
    o2, ls2 = b.attn(causal=False)
    b.lens = full
    ref = b.reference(0, False)
    assert np.abs(o2[0] - ref[0][0]).max() <= b.bounds()[0]


@pytest.mark.parametrize("v_type", [Q4, Q8])
def test_extreme_values(v_type):
    """The largest scales (p * d must stay inside fp16), scores far apart, and
    a long row of almost equal weights."""
    b = Batch([700, 90], [3, 1], H=1, Hq=8, page=64, v_type=v_type, seed=4)
    for kv in b.kv:
        kv[1][:, :, 5] = 65504
        kv[1][:, :, 40] = -65504
    b2 = Batch.__new__(Batch)
    b2.__dict__.update(b.__dict__)
    slots = np.concatenate([b.table[s, np.arange(n) // 64] * 64 + np.arange(n) % 64 for s, n in enumerate(b.lens)])
    kvq.kvq_paged_append(b.pool, *(to_dev(np.concatenate([kv[i] for kv in b.kv])) for i in range(2)), i32(slots))
    b.check()
    b.check(scale=4.0)
    b.q[:] = b.q * 0.001
    b.check()


def test_same_bits_again_and_without_dependent_launch(monkeypatch):
    b = Batch([700, 3000, 40, 1], [60, 1, 40, 1], H=2, Hq=8, page=16, v_type=Q8, seed=5)
    first = b.attn()
    monkeypatch.setenv("KVQ_PDL", "0")
    plain = b.attn()
    monkeypatch.delenv("KVQ_PDL")
    for got in (plain, b.attn(), b.attn(stream=torch.cuda.Stream())):
        assert np.array_equal(first[0], got[0]) and np.array_equal(first[1], got[1])


def test_workspace_is_checked_and_needs_no_preparation():
    b = Batch([700, 40], [3, 1], H=1, Hq=2, page=16, seed=6)
    o = torch.zeros((b.T, 2, 128), device=dev())
    call = kvq.PagedAttnCall(b.pool, to_dev(b.q), i32(b.q_start), 3, i32(b.lens), to_dev(b.table), True, SM_SCALE, o)
    n = call.workspace_size()
    ref = b.attn()
    for fill in (0, 0xFF):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev())
        got = b.attn(workspace=ws)
        assert np.array_equal(ref[0], got[0]) and np.array_equal(ref[1], got[1])
    with pytest.raises(kvq.KvqError) as e:
        b.attn(workspace=torch.empty(n - 1, dtype=torch.uint8, device=dev()))
    assert e.value.status == kvq.KVQ_ERR_WORKSPACE
    with pytest.raises(kvq.KvqError):
        b.attn(workspace=torch.empty(n + 256, dtype=torch.uint8, device=dev())[4:])


@pytest.mark.parametrize("t_q,Hq,H,v_type", [(1, 8, 2, Q4), (4, 8, 1, Q8), (40, 8, 2, Q4)])
def test_agrees_with_segments(t_q, Hq, H, v_type):
    """kvq_decode_attn over the same tokens held in segments."""
    b = Batch([500, 77, 1200], [t_q] * 3, H=H, Hq=Hq, page=32, v_type=v_type, seed=7)
    cache = kvq.Cache(3, H, v_type, max_segs=1)
    for s in range(3):
        cache.add_segment(s, b.lens[s])
        kvq.kvq_append(cache, [s], [b.lens[s]], to_dev(b.kv[s][0]), to_dev(b.kv[s][1]))
    q = to_dev(b.q.reshape(3, t_q, Hq, 128))
    out = torch.empty((3, t_q, Hq, 128), device=dev())
    lse = torch.empty((3, t_q, Hq), device=dev())
    n = kvq.kvq_decode_workspace_size(cache, Hq, t_q, 1200)
    kvq.kvq_decode_attn(cache, q, Hq, t_q, True, i32(b.lens), 1200, None, SM_SCALE, out, lse,
                        torch.empty(n, dtype=torch.uint8, device=dev()) if n else None)
    o, ls = b.attn()
    a, _, el = b.bounds()
    assert np.abs(o - out.cpu().numpy().reshape(o.shape)).max() <= 2 * a
    assert np.abs(ls - lse.cpu().numpy().reshape(ls.shape)).max() <= 2 * el


# ------------------------------------------------------ as a server runs it --
class Server:
    """Fixed buffers of a serving loop: a step is tables, append and attention
    of every layer, all lengths on the GPU."""

    def __init__(self, B, tokens, page=16, n_pages=60, most=12, H=2, Hq=6, v_type=Q4, layers=2, max_q=1):
        d = dev()
        self.page, self.n_pages, self.H, self.Hq, self.v_type, self.tokens = page, n_pages, H, Hq, v_type, tokens
        z = lambda n: torch.zeros(n, dtype=torch.int32, device=d)  # noqa: E731
        self.lens, self.n_new, self.n_free, self.q_start, self.slots, self.status = z(B), z(B), z(1), z(B + 1), z(tokens), z(B)
        self.free = torch.arange(n_pages, dtype=torch.int32, device=d).flip(0).contiguous()
        self.n_free.fill_(n_pages)
        self.table = torch.full((B, most), -1, dtype=torch.int32, device=d)
        self.pools = [kvq.PagePool(n_pages, page, H, v_type) for _ in range(layers)]
        self.qkv = [torch.zeros((tokens, Hq + 2 * H, 128), dtype=torch.float16, device=d) for _ in range(layers)]
        self.out = [torch.zeros((tokens, Hq, 128), dtype=torch.float16, device=d) for _ in range(layers)]
        self.calls = [kvq.PageTablesCall(page, n_pages, self.lens, self.n_new, self.free, self.n_free, self.table, self.lens,
                                         self.n_free, self.q_start, self.slots, self.status)]
        for p, x, o in zip(self.pools, self.qkv, self.out):
            p.data.fill_(POISON)
            self.calls.append(kvq.PagedAppendCall(p, x[:, Hq:Hq + H], x[:, Hq + H:], self.slots))
            self.calls.append(kvq.PagedAttnCall(p, x[:, :Hq], self.q_start, max_q, self.lens, self.table, True, SM_SCALE, o))

    def step(self, stream=None):
        for c in self.calls:
            c(stream)


class Requests:
    """What the server holds, kept on the host."""

    def __init__(self, B, layers, H):
        self.kv = [[[np.zeros((0, H, 128), np.float16)] * 2 for _ in range(layers)] for _ in range(B)]


def _drive(srv, plan, run):
    """plan: per step the n_new of every place; checks each step's rows."""
    r = np.random.default_rng(11)
    B, L, H, Hq = srv.lens.shape[0], len(srv.pools), srv.H, srv.Hq
    held = Requests(B, L, H).kv
    hm = oracle.default_head_map(Hq, H)
    for n_new in plan:
        srv.n_new.copy_(i32(n_new))
        xs = [r.standard_normal((srv.tokens, Hq + 2 * H, 128)).astype(np.float16) for _ in range(L)]
        for x, a in zip(srv.qkv, xs):
            x.copy_(to_dev(a))
        for o in srv.out:
            o.fill_(777)
        run()
        torch.cuda.synchronize()
        assert not srv.status.any()
        t0 = 0
        for b, n in enumerate(n_new):
            if n < 0:
                for lay in range(L):
                    held[b][lay] = [np.zeros((0, H, 128), np.float16)] * 2
                continue
            for lay in range(L):
                rows = xs[lay][t0:t0 + n]
                held[b][lay] = [np.concatenate([held[b][lay][i], rows[:, Hq + i * H:Hq + (i + 1) * H]]) for i in range(2)]
                if n:
                    k, v = held[b][lay]
                    ref = oracle.decode_seq(oracle.quantize_kv(k, v, srv.v_type), rows[:, :Hq], hm, True, SM_SCALE, srv.v_type)
                    got = srv.out[lay][t0:t0 + n].float().cpu().numpy()
                    vmax = np.abs(v.astype(np.float64)).max()
                    # fp16: p * d and the result rounded (2^-11 each), scores as in paged_cases.Batch.bounds
                    assert (np.abs(got - ref["out"]) <= 2.0 ** -11 * (vmax + np.abs(ref["out"])) + 4e-4).all()
            t0 += max(n, 0)
        assert srv.lens.cpu().tolist() == [len(held[b][0][0]) for b in range(B)]
        for o in srv.out:
            assert (o[t0:] == 777).all()


def test_steps_in_a_row():
    """Prompts in chunks, decodes, ends, places taken again."""
    srv = Server(5, 64, max_q=40)
    _drive(srv, [[40, 7, 0, 16, 1], [33, 1, 30, 0, 0], [1, 1, 1, 1, 1], [-1, 1, 1, -1, 1], [20, 1, 1, 17, 1], [1, 1, -1, 1, 1],
                 [1, -1, 12, 1, 33], [1, 1, 1, 1, 1]], srv.step)
    used = (-(-srv.lens // srv.page)).sum()
    assert int(srv.n_free) == srv.n_pages - int(used)
    # no page is listed twice
    t, n = srv.table.cpu().numpy(), srv.lens.cpu().numpy()
    pages = np.concatenate([t[b, :-(-n[b] // srv.page)] for b in range(5)] + [srv.free.cpu().numpy()[:int(srv.n_free)]])
    assert np.array_equal(np.sort(pages), np.arange(srv.n_pages))


def test_steps_replayed_from_a_graph():
    """One captured step, replayed while the lengths grow on the device."""
    srv = Server(6, 24, max_q=9)
    s = torch.cuda.Stream()
    srv.step(s)               # first use outside the capture (n_new = 0: nothing changes)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        srv.step(s)
    _drive(srv, [[9, 1, 5, 0, 8, 1], [1, 9, 1, 1, 1, 1], [9, 1, 1, 1, 3, 9]] + [[1] * 6] * 3 + [[-1, 1, 1, -1, 1, 1], [9, 1, 1, 5, 1, 1]],
           g.replay)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each."""
    bs = [Batch([900, 40, 1500], [1, 30, 2], H=2, Hq=8, page=16, seed=s) for s in (1, 2)]
    want = [b.attn() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    outs, calls = [], []
    for b in bs:
        o = torch.zeros((b.T, 8, 128), device=dev())
        outs.append(o)
        calls.append(kvq.PagedAttnCall(b.pool, to_dev(b.q), i32(b.q_start), 30, i32(b.lens), to_dev(b.table), True, SM_SCALE, o))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.cpu().numpy().astype(np.float64), w[0])
