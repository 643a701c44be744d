"""What surrounds the paged cache's append and attention, on a GPU: each operator
of include/kvq_tokens.h against its formula in 64 bits or plain Python, at the
sizes, layouts and values where it can go wrong."""
import numpy as np
import pytest
import torch

import oracle
from quantized_kv_cache_03_gb300 import kvq

from kvq_cases import SM_SCALE, dev
from paged_cases import POISON, i32, pool_rows, to_dev, values
from tokens_cases import FP32, fork_ref, fp16_bound, normalized, rates, rotated

pytestmark = pytest.mark.gpu

I8, F16 = kvq.K_I8, kvq.K_F16
Q4, Q8 = kvq.V_Q4_0, kvq.V_Q8_0
HALF, PAIRS = kvq.ROPE_HALF, kvq.ROPE_PAIRS
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def near16(got, y, size, what=""):
    d = np.abs(f64(got) - y)
    bad = d > fp16_bound(y, size)
    assert not bad.any(), "%s off by %.3g at %s, allowed %.3g" % (what, d[bad].max(), np.argwhere(bad)[0], fp16_bound(y, size)[bad].min())


# ------------------------------------------------------------- positions --
@pytest.mark.parametrize("new,pad", [([1], 0), ([1] * 4096, 0), ([0, 5, 0, 0, 300, 1, 0], 9), ([], 5), ([0, 0], 3), ([1023, 1, 1025, 2], 0), ([7] * 300, 4000)])
def test_positions(new, pad):
    r = np.random.default_rng(len(new))
    lens = [n + int(r.integers(0, 100000)) for n in new]
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = i32(np.full(sum(new) + pad + 1, 99))
    kvq.kvq_page_positions(i32(qs), i32(lens), out[:-1])
    want = [np.arange(L - n, L) for L, n in zip(lens, new)] + [np.full(pad, -1), [99]]
    assert np.array_equal(out.cpu().numpy(), np.concatenate(want))


def test_positions_hold_bad_row_ranges():
    out = i32(np.full(10, 99))
    kvq.kvq_page_positions(i32([-5, 3, 2 ** 31 - 1]), i32([10, 20]), out[:8])
    assert out.tolist() == [7, 8, 9, 15, 16, 17, 18, 19, 99, 99]


# ---------------------------------------------------------- new tokens in --
def _tokens(r, T, Hq, H, big=False):
    x = r.standard_normal((T, Hq + 2 * H, 128))
    if big:
        x *= np.exp2(r.uniform(-12, 9, (T, Hq + 2 * H, 1)))
    return x.astype(np.float16)


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("n_rot", [128, 64, 40, 8, 0])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,Hq,H", [(1, 1, 1), (2, 5, 1), (33, 3, 2), (130, 7, 8)])
def test_normalized_and_rotated(T, Hq, H, norm, n_rot, layout):
    """Queries and keys left as fp16, from strided rows and in place."""
    r = np.random.default_rng(T + n_rot)
    x = _tokens(r, T, Hq, H, big=True)
    pos = r.integers(0, 1 << 20, T)
    pos[:1] = 0
    kw = dict(scaling=kvq.ROPE_BY_INDEX, factor=8.0, original=4096.0, fast=32.0, slow=1.0)
    rope = kvq.Rope(n_rot, 10000.0, layout, device=dev(), **kw)
    f, amp = rates(n_rot, 10000.0, **kw)
    wq, wk = ((1 + r.standard_normal(128)).astype(np.float32) if norm else None for _ in range(2))
    w = [None if a is None else to_dev(a) for a in (wq, wk)]
    want = [rotated(normalized(x[:, a:b], wt, EPS), pos, f, amp, layout) for a, b, wt in ((0, Hq, wq), (Hq, Hq + H, wk))]
    outs = []
    for in_place in (False, True):
        t = to_dev(x)
        q, k = t[:, :Hq], t[:, Hq:Hq + H]
        qo = q if in_place else torch.full((T, Hq, 128), 777.0, dtype=torch.float16, device=dev())
        ko = k if in_place else torch.full((T, H + 1, 128), 777.0, dtype=torch.float16, device=dev())[:, 1:]
        kvq.kvq_qkv(q, k, None, i32(pos), rope, qo, k_out=ko, q_norm=w[0], k_norm=w[1], eps=EPS)
        for got, (y, size), what in ((qo, want[0], "q"), (ko, want[1], "k")):
            near16(got, y, size, what)
        outs.append((qo.clone(), ko.clone()))
        if in_place:
            assert np.array_equal(t[:, Hq + H:].cpu().numpy(), x[:, Hq + H:])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("layout", [HALF, PAIRS])
def test_far_and_negative_positions(layout):
    pos = np.array([0, 1, -1, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789])
    r = np.random.default_rng(1)
    x = _tokens(r, len(pos), 2, 0)
    f, _ = rates(128, 500000.0)
    out = torch.zeros((len(pos), 2, 128), dtype=torch.float16, device=dev())
    kvq.kvq_qkv(to_dev(x), None, None, i32(pos), kvq.Rope(128, 500000.0, layout, device=dev()), out)
    # the reference's own angle: a rate known to 2^-52 of itself (power and product), times the position; and half a unit of 2^-64 turns a position
    y, size = rotated(x.astype(np.float64), pos, f, 1.0, layout)
    extra = (np.abs(pos)[:, None, None] * (4 * 2.0 ** -52 + 2 ** -64 * 2 * np.pi)) * size
    assert (np.abs(f64(out) - y) <= fp16_bound(y, size) + extra).all()


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("layout,n_rot,norm", [(HALF, 128, True), (PAIRS, 128, False), (HALF, 24, False), (PAIRS, 64, True), (HALF, 0, True)])
@pytest.mark.parametrize("T,Hq,H,page", [(1, 4, 1, 16), (37, 6, 2, 32), (260, 8, 8, 64), (9, 0, 3, 256)])
def test_into_pages(T, Hq, H, page, layout, n_rot, norm, k_type, v_type):
    """The bytes are those of the fp16 keys appended; nothing else of the pool changes.  Runs of slots from odd places, scattered ones, backwards."""
    r = np.random.default_rng(T)
    x = to_dev(_tokens(r, T, Hq, H, big=True))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    n_pages = -(-T // page) + 2
    pos, rope = i32(r.integers(0, 100000, T)), kvq.Rope(n_rot, layout=layout, device=dev())
    w = to_dev((1 + 0.3 * r.standard_normal((2, 128))).astype(np.float32)) if norm else [None, None]
    qp, kp = torch.zeros((T, max(1, Hq), 128), dtype=torch.float16, device=dev())[:, :Hq], torch.zeros((T, H, 128), dtype=torch.float16, device=dev())
    queries = dict(q16=q, q_out=qp) if Hq else dict(q16=None, q_out=None)
    kvq.kvq_qkv(k16=k, v16=None, positions=pos, rope=rope, k_out=kp, q_norm=w[0], k_norm=w[1], **queries)
    for order in ("runs", "odd", "scattered", "backwards"):
        slots = page // 2 + np.arange(T) + (order == "odd")
        slots = r.permutation(n_pages * page)[:T] if order == "scattered" else slots[::-1].copy() if order == "backwards" else slots
        one, two = (kvq.PagePool(n_pages, page, H, v_type, k_type=k_type) for _ in range(2))
        one.data.fill_(POISON)
        two.data.fill_(POISON)
        qo = torch.zeros_like(qp)
        queries = dict(q16=q, q_out=qo) if Hq else dict(q16=None, q_out=None)
        kvq.kvq_qkv(k16=k, v16=v, positions=pos, rope=rope, pool=one, slots=i32(slots), q_norm=w[0], k_norm=w[1], **queries)
        kvq.kvq_paged_append(two, kp.contiguous(), v.contiguous(), i32(slots))
        assert torch.equal(one.data, two.data), order
        assert torch.equal(qo, qp), order


def test_rows_left_out():
    """Negative slots leave a token out; slots past the pool only its key and value."""
    T, Hq, H = 9, 3, 2
    r = np.random.default_rng(4)
    x = to_dev(_tokens(r, T, Hq, H))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    slots = [-1, 5, 32, -2 ** 31, 2 ** 31 - 1, 6, 7, -1, 33]
    pos, rope = i32(np.arange(T)), kvq.Rope(128, device=dev())
    pool = kvq.PagePool(2, 16, H, Q8)
    pool.data.fill_(POISON)
    qo = torch.full((T, Hq, 128), 777.0, dtype=torch.float16, device=dev())
    kvq.kvq_qkv(q, k, v, pos, rope, qo, pool=pool, slots=i32(slots))
    qa, ka, kb = torch.zeros_like(qo), torch.zeros((T, H, 128), dtype=torch.float16, device=dev()), torch.full((T, H, 128), 777.0, dtype=torch.float16, device=dev())
    kvq.kvq_qkv(q, k, None, pos, rope, qa, k_out=ka)
    kvq.kvq_qkv(None, k, None, pos, rope, None, k_out=kb, slots=i32(slots))
    for t, s in enumerate(slots):
        assert torch.equal(qo[t], qa[t]) if s >= 0 else (qo[t] == 777).all()
        assert torch.equal(kb[t], ka[t]) if s >= 0 else (kb[t] == 777).all()
    want = kvq.PagePool(2, 16, H, Q8)
    want.data.fill_(POISON)
    kvq.kvq_paged_append(want, ka, v.contiguous(), i32(slots))
    assert torch.equal(pool.data, want.data)


@pytest.mark.parametrize("T", [1, 40, 700, 3700])
def test_in_place_into_pages(T):
    """A fused projection's output whose queries turn where they lie, captured and replayed; keys, values and the rows of
    tokens that are left out stay as they are."""
    Hq, H, page = 5, 2, 32
    r = np.random.default_rng(T)
    x = to_dev(_tokens(r, T, Hq, H))
    n_pages = -(-T // page) + 1
    slots = np.where(r.random(T) < 0.3, -1, np.arange(T) + 7)
    slots[-(T // 3):] = -1 if T > 2 else slots[0]
    slots, pos, rope = i32(slots), i32(r.integers(0, 99999, T)), kvq.Rope(128, device=dev())
    w = to_dev(r.standard_normal(128).astype(np.float32))
    pools = [kvq.PagePool(n_pages, page, H, Q4) for _ in range(2)]
    want = x[:, :Hq].clone()
    for p in pools:
        p.data.fill_(POISON)
    kvq.kvq_qkv(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], pos, rope, want, pool=pools[0], slots=slots, q_norm=w)
    y = x.clone()
    call = kvq.QkvCall(y[:, :Hq], y[:, Hq:Hq + H], y[:, Hq + H:], pos, rope, y[:, :Hq], pool=pools[1], slots=slots, q_norm=w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        y.copy_(x)
        pools[1].data.fill_(POISON)
        graph.replay()
        assert torch.equal(y[:, :Hq], want) and torch.equal(y[:, Hq:], x[:, Hq:]) and torch.equal(pools[0].data, pools[1].data)
    assert torch.equal(want[slots < 0], x[:, :Hq][slots < 0])


def test_values_that_are_not_finite_and_large_ones():
    """A head that holds an infinity or NaN is its own affair; values that do not rotate are not touched by it."""
    r = np.random.default_rng(5)
    x = _tokens(r, 4, 3, 0)
    x[0, 1, 3], x[1, 2, 100], x[2, 0, 70], x[3, 1, 127] = np.inf, np.nan, -np.inf, 65504
    for layout in (HALF, PAIRS):
        for norm in (None, torch.ones(128, device=dev())):
            out = torch.zeros((4, 3, 128), dtype=torch.float16, device=dev())
            kvq.kvq_qkv(to_dev(x), None, None, i32([3, 4, 5, 6]), kvq.Rope(64, layout=layout, device=dev()), out, q_norm=norm, eps=EPS)
            o = f64(out)
            bad = np.zeros((4, 3), bool)
            bad[0, 1] = bad[1, 2] = bad[2, 0] = True
            y, size = rotated(normalized(np.where(bad[..., None], 1, x), None if norm is None else np.ones(128), EPS), [3, 4, 5, 6], rates(64)[0], 1.0, layout)
            assert (np.abs(o - y) <= fp16_bound(y, size))[~bad].all()
            if norm is None:
                assert o[1, 2, 99] == x[1, 2, 99] and np.isnan(o[1, 2, 100]) and o[2, 0, 70] == -np.inf and o[2, 0, 71] == x[2, 0, 71]
                assert np.isfinite(o[0, 1, 64:]).all() and not np.isfinite(o[0, 1, 3])
            else:
                assert np.isnan(o[bad]).any(-1).all()


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
def test_quantized_as_append_does(k_type, v_type):
    """Values at, just below and just above the halves of their scale, at scales from fp16's subnormals to its largest, zeros,
    infinities and NaN among them: the bytes of kvq_paged_append, from pairs of places and single ones."""
    r = np.random.default_rng(3)
    n, H = 256, 4
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
        x[23, :, 2] = np.nan
        kv.append(to_dev(np.ascontiguousarray(x.reshape(n, H, 128))))
    ka = torch.zeros_like(kv[0])
    kvq.kvq_qkv(None, kv[0], None, None, None, None, k_out=ka)   # the fp16 keys: as they were, NaN with bits of its own
    assert torch.equal(torch.nan_to_num(ka), torch.nan_to_num(kv[0])) and torch.equal(ka.isnan(), kv[0].isnan())
    for slots in (np.arange(n), np.arange(n) + 7, 2 * np.arange(n) % 509):
        one, two = (kvq.PagePool(9, 64, H, v_type, k_type=k_type) for _ in range(2))
        one.data.fill_(POISON)
        two.data.fill_(POISON)
        kvq.kvq_qkv(None, kv[0], kv[1], None, None, None, pool=one, slots=i32(slots))
        kvq.kvq_paged_append(two, ka, kv[1], i32(slots))
        assert torch.equal(one.data, two.data)


def test_into_pages_past_32_bits():
    H, page = 8, 256
    n_pages = (5 << 30) // (H * 16 * 4352)
    pool = kvq.PagePool(n_pages, page, H, Q8)
    r = np.random.default_rng(8)
    x = to_dev(_tokens(r, 20, 1, H))
    slots = np.concatenate([np.arange(10) + (n_pages - 1) * page + 3, np.arange(10)])
    rope, pos, q = kvq.Rope(128, device=dev()), i32(np.arange(20) + 9), torch.zeros((20, 1, 128), dtype=torch.float16, device=dev())
    kvq.kvq_qkv(x[:, :1], x[:, 1:1 + H], x[:, 1 + H:], pos, rope, q, pool=pool, slots=i32(slots))
    small, ka = kvq.PagePool(2, page, H, Q8), torch.zeros((20, H, 128), dtype=torch.float16, device=dev())
    kvq.kvq_qkv(None, x[:, 1:1 + H], None, pos, rope, None, k_out=ka)
    kvq.kvq_paged_append(small, ka, x[:, 1 + H:].contiguous(), i32(np.where(slots >= page, slots - (n_pages - 2) * page, slots)))
    outs = [torch.zeros((20, H, 128), device=dev()) for _ in range(4)]
    kvq.kvq_paged_gather(pool, i32(slots), outs[0], outs[1])
    kvq.kvq_paged_gather(small, i32(np.where(slots >= page, slots - (n_pages - 2) * page, slots)), outs[2], outs[3])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3]) and outs[0].any()


def test_a_large_step():
    """More tokens and heads than one pass of the launch holds."""
    T, Hq, H = 5001, 20, 4
    r = np.random.default_rng(6)
    x = _tokens(r, T, Hq, H)
    pos = r.integers(0, 32768, T)
    t = to_dev(x)
    qo = torch.zeros((T, Hq, 128), dtype=torch.float16, device=dev())
    pool = kvq.PagePool(-(-T // 64), 64, H, Q4)
    kvq.kvq_qkv(t[:, :Hq], t[:, Hq:Hq + H], t[:, Hq + H:], i32(pos), kvq.Rope(128, device=dev()), qo, pool=pool, slots=i32(np.arange(T)))
    y, size = rotated(x[:, :Hq].astype(np.float64), pos, rates(128)[0], 1.0, HALF)
    near16(qo, y, size)
    y, size = rotated(x[:, Hq:Hq + H].astype(np.float64), pos, rates(128)[0], 1.0, HALF)
    rows = pool_rows(pool)
    k = values({n: a.transpose(0, 2, 1, 3).reshape(-1, H, a.shape[-1])[:T] for n, a in rows.items()}, Q4)[0]
    step = np.repeat(rows["ks"].transpose(0, 2, 1, 3).reshape(-1, H, 4)[:T].copy().view(np.float16).astype(np.float64), 32, -1)
    assert (np.abs(k - y) <= fp16_bound(y, size) + 0.5 * step * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("T,Hq,H", [(3650, 9, 3), (3900, 12, 2), (7301, 3, 5), (11000, 4, 1)])
def test_a_large_step_is_its_parts(T, Hq, H):
    """The bits do not depend on how the launch deals out tokens and heads: one call, and calls of some tokens each."""
    r = np.random.default_rng(T)
    page, part = 32, 611
    n_pages = -(-T // page) + 3
    t = to_dev(_tokens(r, T, Hq, H))
    order = np.concatenate([np.arange(1, T // 2), r.permutation(np.arange(T // 2, n_pages * page))])[:T]   # neighbours, and none
    slots = np.where(r.random(T) < 0.1, np.where(r.random(T) < 0.5, -1, n_pages * page + 5), order)
    pos, w = i32(r.integers(0, 131072, T)), to_dev(r.standard_normal(128).astype(np.float32))
    rope, slots = kvq.Rope(128, device=dev()), i32(slots)
    got = []
    for step in (T, part):
        q, pool = torch.full((T, Hq, 128), 3.0, dtype=torch.float16, device=dev()), kvq.PagePool(n_pages, page, H, Q8)
        pool.data.fill_(0)
        for a in range(0, T, step):
            b = slice(a, a + step)
            kvq.kvq_qkv(t[b, :Hq], t[b, Hq:Hq + H], t[b, Hq + H:], pos[b], rope, q[b], pool=pool, slots=slots[b], q_norm=w, k_norm=w)
        got.append((q, pool.data))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])


# ------------------------------------------------------------------ fork --
def _fork_state(r, B, page, most, extra, hi, group=1, hidden=0.0):
    """Old tables of groups whose members share whole pages of a prefix."""
    lens, table, pages = np.zeros(B, np.int64), np.full((B, most), -9, np.int32), 0
    for g in range(0, B, group):
        shared = int(r.integers(0, hi // page + 1))
        first = list(range(pages, pages + shared))
        pages += shared
        for b in range(g, min(B, g + group)):
            n = int(r.integers(0, hi + 1))
            blocks = -(-n // page)
            row = first[:blocks] + list(range(pages, pages + max(0, blocks - shared)))
            pages += max(0, blocks - shared)
            lens[b] = n
            table[b, :blocks] = row
    n_pages = pages + extra
    ids = r.permutation(n_pages).astype(np.int32)
    table = np.where(table >= 0, ids[np.maximum(table, 0)], table).astype(np.int32)
    if hidden:
        table = np.where(r.random(table.shape) < hidden, np.where(r.random(table.shape) < 0.5, n_pages + 3, -1), table).astype(np.int32)
    free = np.full(n_pages, -5, np.int32)
    free[:extra] = ids[pages:]
    return lens, table, free, extra, n_pages


def _run_fork(page, n_pages, lens, table, free, n_free, most, parent=None, keep=None, in_place=False, same_table=False, pad=0):
    B = len(lens)
    wide = np.full((B, table.shape[1] + pad), -77, np.int32)
    wide[:, :table.shape[1]] = table
    d = dict(lens=i32(lens), table=to_dev(wide)[:, :most], free=to_dev(free), n_free=i32([n_free]))
    out = torch.full((B, most + pad), -8, dtype=torch.int32, device=dev())
    o = dict(table_out=d["table"] if same_table else out[:, :most], lens=d["lens"] if in_place else i32(np.full(B, 99)),
             n_free=d["n_free"] if in_place else i32([99]), **{k: i32(np.full(B, 99)) for k in ("copy_from", "copy_to", "copy_held", "status")})
    kvq.kvq_page_fork(page, n_pages, d["lens"], d["table"], d["free"], d["n_free"], o["table_out"], o["lens"], o["n_free"], o["copy_from"],
                      o["copy_to"], o["copy_held"], o["status"], parent=None if parent is None else i32(parent), keep=None if keep is None else i32(keep))
    torch.cuda.synchronize()
    assert (out[:, most:] == -8).all()
    if not same_table:
        assert np.array_equal(d["table"].cpu().numpy(), table[:, :most])
    return dict(o, free=d["free"])


def _same(got, ref):
    for k, v in ref.items():
        g = got[k].cpu().numpy()
        assert np.array_equal(g, v), "%s differs at %s: %s, not %s" % (k, np.argwhere(g != v)[:4].tolist(), g[g != v][:4], np.asarray(v)[g != v][:4])


@pytest.mark.parametrize("B,page,hi,group,extra", [(1, 16, 40, 1, 3), (4, 16, 70, 4, 5), (40, 64, 900, 4, 50), (256, 16, 300, 8, 300), (1000, 32, 100, 2, 1100),
                                                   (4096, 16, 20, 4, 4200), (6, 256, 70000, 3, 40), (3, 16, 30000, 1, 1)])
def test_fork(B, page, hi, group, extra):
    r = np.random.default_rng(B)
    most = -(-hi // page) + 1
    lens, table, free, n_free, n_pages = _fork_state(r, B, page, most, extra, hi, group)
    everyone = np.arange(B)
    near = (everyone // group) * group + r.integers(0, group, B)
    near = np.minimum(near, B - 1)
    for parent, keep in ((None, None), (near, None), (r.integers(0, B, B), r.integers(-3, hi + 50, B)), (np.where(r.random(B) < 0.4, -1, near), lens[near] - r.integers(0, 20, B)),
                         (np.full(B, B - 1), None), (np.full(B, B), None), (r.permutation(B), np.full(B, 2 ** 31 - 1)), (None, lens - 1), (None, np.zeros(B))):
        ref = fork_ref(page, n_pages, lens, table, free, n_free, np.full((B, most), -8, np.int32), most, parent, keep)
        for kw in (dict(), dict(in_place=True, pad=3)):
            _same(_run_fork(page, n_pages, lens, table, free, n_free, most, parent, keep, **kw), ref)
        if parent is None:
            ref = fork_ref(page, n_pages, lens, table, free, n_free, table[:, :most], most, parent, keep)
            _same(_run_fork(page, n_pages, lens, table, free, n_free, most, parent, keep, in_place=True, same_table=True), ref)


def test_fork_of_nothing():
    ref = fork_ref(16, 4, [], np.zeros((0, 2), np.int32), np.arange(4, dtype=np.int32), 3, np.zeros((0, 2), np.int32), 2)
    _same(_run_fork(16, 4, np.zeros(0, int), np.zeros((0, 2), np.int32), np.arange(4, dtype=np.int32), 3, 2), ref)
    lens, table = np.array([5, 0]), np.zeros((2, 0), np.int32)
    ref = fork_ref(16, 4, lens, table, np.arange(4, dtype=np.int32), 3, table, 0)
    _same(_run_fork(16, 4, lens, table, np.arange(4, dtype=np.int32), 3, 0), ref)
    free = np.zeros(0, np.int32)
    lens, table = np.array([5, 0]), np.full((2, 1), 3, np.int32)
    _same(_run_fork(16, 0, lens, table, free, 3, 1), fork_ref(16, 0, lens, table, free, 3, np.full((2, 1), -8, np.int32), 1))


@pytest.mark.parametrize("seed", range(5))
def test_fork_short_of_pages_and_with_hidden_ones(seed):
    """Too few pages for the copies; entries outside the pool; lengths and a stack size out of range; a page that two rows list in different places."""
    r = np.random.default_rng(seed)
    B, page, most = 60, 16, 9
    lens, table, free, n_free, n_pages = _fork_state(r, B, page, most, [0, 3, 10, 40, 2][seed], 130, 4, hidden=0.1 * (seed % 3))
    lens = lens.copy()
    lens[3], lens[7] = -4, 10 ** 6
    table[9, :3] = table[10, [2, 0, 1]]
    table[11, 0] = table[11, 1]      # the same page twice in a row
    parent, keep = r.integers(-1, B + 1, B), r.integers(0, 140, B)
    for given in (n_free, -5, 10 ** 6):
        ref = fork_ref(page, n_pages, lens, table, free, given, np.full((B, most), -8, np.int32), most, parent, keep)
        _same(_run_fork(page, n_pages, lens, table, free, given, most, parent, keep), ref)


@pytest.mark.parametrize("left", [0, 1, 7, 58, 59])
def test_fork_of_one_place_into_all(left):
    """59 copies of a last page wanted, `left` pages there: the first places get theirs, the others keep their whole pages."""
    B, page, most, n_pages = 60, 16, 4, 70
    lens, table = np.zeros(B, np.int64), np.full((B, most), -9, np.int32)
    lens[5], table[5, :3] = 40, [61, 2, 33]
    free = np.full(n_pages, -5, np.int32)
    free[:left] = np.arange(left) % 28 + 3
    ref = fork_ref(page, n_pages, lens, table, free, left, np.full((B, most), -8, np.int32), most, np.full(B, 5))
    assert ref["status"].sum() == 59 - left and (ref["lens"] == 32).sum() == 59 - left
    _same(_run_fork(page, n_pages, lens, table, free, left, most, np.full(B, 5)), ref)


@pytest.mark.parametrize("B,n_pages", [(1, 5), (3, 0), (200, 40), (1024, 7), (1500, 40)])
def test_fork_of_rows_without_entries(B, n_pages):
    """A table of no columns: every length is held to 0, nothing is copied or given back."""
    lens, free = np.arange(B) % 50, np.arange(n_pages, dtype=np.int32)
    table = np.zeros((B, 0), np.int32)
    for parent, keep in ((None, None), (np.arange(B)[::-1].copy(), np.full(B, 3))):
        ref = fork_ref(16, n_pages, lens, table, free, n_pages // 2, table, 0, parent, keep)
        assert not ref["lens"].any() and not ref["status"].any()
        _same(_run_fork(16, n_pages, lens, table, free, n_pages // 2, 0, parent, keep), ref)


def test_fork_over_a_large_pool():
    """A million pages, most of them in no list."""
    r = np.random.default_rng(8)
    B, page, most, n_pages = 50, 16, 2000, 1_000_003
    ids = r.permutation(n_pages).astype(np.int32)
    lens = r.integers(0, most * page + 1, B)
    table = ids[:B * most].reshape(B, most).copy()
    free = np.full(n_pages, -5, np.int32)
    free[:500_000] = ids[B * most:B * most + 500_000]
    parent = r.integers(-10, B, B)
    ref = fork_ref(page, n_pages, lens, table, free, 500_000, np.full((B, most), -8, np.int32), most, parent)
    _same(_run_fork(page, n_pages, lens, table, free, 500_000, most, parent), ref)


# ------------------------------------------------------------------ copy --
@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (F16, Q8)])
@pytest.mark.parametrize("page,H,n,pools", [(16, 1, 1, 1), (64, 3, 5, 2), (256, 8, 20, 1), (32, 2, 300, 7), (16, 1, 2, 128)])
def test_copy(page, H, n, pools, k_type, v_type):
    r = np.random.default_rng(n)
    n_pages = 2 * n + 2
    ps = [kvq.PagePool(n_pages, page, H, v_type, k_type=k_type) for _ in range(pools)]
    for p in ps:
        p.data.random_(0, 256)
    before = [p.data.cpu().numpy().reshape(n_pages, H, page // 16, -1) for p in ps]
    ids = r.permutation(n_pages)
    for held in (None, r.integers(-5, page + 40, n)):
        frm, to = ids[:n].copy(), ids[n:2 * n].copy()
        if n > 4:
            frm[1] = frm[0]                                      # a page copied to two
            frm[2], to[3], to[4] = -1, n_pages, frm[4]           # pairs that name no two pages
        kvq.kvq_page_copy(ps, i32(frm), i32(to), held=None if held is None else i32(held))
        for p, b in zip(ps, before):
            for i in range(n):
                if frm[i] >= 0 and to[i] < n_pages:
                    t = page // 16 if held is None else -(-min(max(held[i], 0), page) // 16)
                    b[to[i], :, :t] = b[frm[i], :, :t]
            assert np.array_equal(p.data.cpu().numpy().reshape(b.shape), b)


def test_copy_in_pools_of_several_kinds():
    r = np.random.default_rng(0)
    kinds = [(1, I8, Q4), (5, F16, Q8), (2, I8, Q8), (3, F16, Q4)]
    ps = [kvq.PagePool(9, 32, H, v, k_type=k) for H, k, v in kinds]
    for p in ps:
        p.data.random_(0, 256)
    before = [p.data.cpu().numpy().reshape(9, -1) for p in ps]
    kvq.kvq_page_copy(ps, i32([0, 4, 7]), i32([8, 2, 1]))
    for p, b in zip(ps, before):
        b[[8, 2, 1]] = b[[0, 4, 7]]
        assert np.array_equal(p.data.cpu().numpy().reshape(9, -1), b)


def test_copy_past_32_bits():
    """Pages whose bytes lie more than 4 GB into the pool."""
    H, page = 8, 256
    n_pages = (5 << 30) // (H * 16 * 4352)
    pool = kvq.PagePool(n_pages, page, H, Q8)
    bytes_ = pool.data.view(n_pages, -1)
    bytes_[0].random_(0, 256)
    bytes_[n_pages - 2].random_(0, 256)
    kvq.kvq_page_copy([pool], i32([0, n_pages - 2]), i32([n_pages - 1, 1]))
    assert torch.equal(bytes_[0], bytes_[n_pages - 1]) and torch.equal(bytes_[n_pages - 2], bytes_[1])
    # and tokens of theirs moved, whole and turned
    slot = (n_pages - 1) * page
    kvq.kvq_paged_move(pool, i32([slot + 7]), i32([2 * page + 3]), staged=True)
    kvq.kvq_paged_move(pool, i32([3]), i32([slot + 9]), staged=False)
    tiles = bytes_.view(n_pages, H, page // 16, -1)[[0, 2, n_pages - 1]].cpu().numpy()
    from paged_cases import split_tiles
    rows = split_tiles(tiles, I8, Q8)
    for a in rows.values():
        assert np.array_equal(a[1, :, 0, 3], a[0, :, 0, 7]) and np.array_equal(a[2, :, 0, 9], a[0, :, 0, 3])


# ---------------------------------------------------------------- gather --
@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("T,H,page", [(4096, 1, 16), (1370, 3, 64), (513, 8, 256), (5001, 8, 32)])
def test_gather_of_many_rows(T, H, page, k_type, v_type):
    """Rows past the size from which a warp takes eight: exact values (code * scale fits 24 bits), rounded once in fp16; slots in
    order, scattered, listed twice, and ones that are none, whose rows stay."""
    r = np.random.default_rng(T)
    n_pages = 700 // page + 3
    pool, rows = _filled(r, n_pages, page, H, k_type, v_type)
    k, v = values(rows, v_type)
    slots = r.integers(0, n_pages * page, T)
    slots[:200] = np.arange(200) + 5
    slots[r.integers(0, T, 40)] = -1
    slots[7:9] = n_pages * page, 2 ** 31 - 1
    slots[-1] = -2 ** 31
    some = (slots >= 0) & (slots < n_pages * page)
    for dt, npt in ((torch.float32, np.float32), (torch.float16, np.float16)):
        ko, vo = (torch.full((T, H, 128), 777.0, dtype=dt, device=dev()) for _ in range(2))
        kvq.kvq_paged_gather(pool, i32(slots), ko, vo)
        for o, ref in ((ko, k), (vo, v)):
            want = np.full((T, H, 128), 777, npt)
            with np.errstate(over="ignore"):
                want[some] = ref[slots[some]].astype(npt)
            assert np.array_equal(o.cpu().numpy(), want)


# ------------------------------------------------------------------ move --
def _filled(r, n_pages, page, H, k_type, v_type, big=True):
    """A pool of quantized tokens, and its rows."""
    pool = kvq.PagePool(n_pages, page, H, v_type, k_type=k_type)
    T = n_pages * page
    kv = r.standard_normal((2, T, H, 128))
    if big:
        kv *= np.exp2(r.uniform(-9, 9, (2, T, H, 1)))
    kv[0, 3, 0, 32:64] = 0     # a block of zeros
    kv = kv.astype(np.float16)
    kvq.kvq_paged_append(pool, to_dev(kv[0]), to_dev(kv[1]), i32(np.arange(T)))
    return pool, _by_slot(pool)


def _by_slot(pool):
    return {n: a.transpose(0, 2, 1, 3).reshape(-1, pool.n_kv_heads, a.shape[-1]) for n, a in pool_rows(pool).items()}


def _moves(r, kind, S, n):
    if kind == "down":          # a stretch moves down by an odd number of places, over itself
        return np.arange(n) + 5, np.arange(n)
    if kind == "up":
        return np.arange(n), np.arange(n) + 2
    if kind == "mixed":
        return r.permutation(S)[:n], r.permutation(S)[:n]
    if kind == "reversed":
        return np.arange(n), np.arange(n)[::-1].copy()
    p = r.permutation(S)        # apart: no slot is read and written
    return p[:n], np.sort(p[n:2 * n])


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("page,H,n", [(16, 1, 1), (16, 2, 13), (64, 3, 150), (256, 8, 300)])
@pytest.mark.parametrize("kind", ["down", "up", "mixed", "reversed", "apart"])
def test_moved_bytes(kind, page, H, n, k_type, v_type):
    r = np.random.default_rng(n)
    n_pages = -(-2 * n // page) + 1
    pool, rows = _filled(r, n_pages, page, H, k_type, v_type)
    frm, to = _moves(r, kind, n_pages * page, n)
    bad = np.array([[-1, 0], [0, -7], [n_pages * page, 1], [1, 2 ** 31 - 1]])       # tokens without a slot
    bad = bad[[int(b[1]) not in to or not 0 <= b[0] < n_pages * page or not 0 <= b[1] < n_pages * page for b in bad]]
    f2, t2 = np.concatenate([frm[:n // 2], bad[:, 0], frm[n // 2:]]), np.concatenate([to[:n // 2], bad[:, 1], to[n // 2:]])
    ways = [dict(staged=True)] + ([dict(staged=False)] if kind == "apart" else [])
    start = pool.data.clone()
    for way in ways:
        for rope in (dict(), dict(rope=kvq.Rope(128, device=dev()), turn=i32(np.zeros(len(f2))))):
            pool.data.copy_(start)
            kvq.kvq_paged_move(pool, i32(f2), i32(t2), **way, **rope)
            got = _by_slot(pool)
            for name, a in rows.items():
                want = a.copy()
                want[to] = a[frm]
                assert np.array_equal(got[name], want), (name, way)


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("turned", [False, True])
def test_some_stay_and_some_move(turned, k_type, v_type):
    """Pairs of neighbouring slots of which one's token stays where it is and the other's comes from elsewhere."""
    r = np.random.default_rng(7)
    page, H, n = 32, 3, 60
    pool, rows = _filled(r, 6, page, H, k_type, v_type)
    to = np.arange(n) + 1
    frm = np.where(r.random(n) < 0.5, to, 100 + r.permutation(90)[:n])
    turn = np.where(r.random(n) < 0.5, 0, r.integers(-99, 99, n)) if turned else np.zeros(n, int)
    kvq.kvq_paged_move(pool, i32(frm), i32(to), rope=kvq.Rope(128, device=dev()) if turned else None, turn=i32(turn) if turned else None, staged=False)
    got = _by_slot(pool)
    for name, a in rows.items():
        want, same = a.copy(), np.ones(len(a), bool)
        want[to] = a[frm]
        if name in ("kq", "ks", "k16"):
            same[to[turn != 0]] = False
        assert np.array_equal(got[name][same], want[same]), name
    k0, k1 = values(rows, v_type)[0], values(got, v_type)[0]
    y, size = rotated(k0[frm], turn, rates(128)[0], 1.0, HALF)
    allowed = fp16_bound(y, size)
    if k_type == I8:
        allowed = allowed + 0.5 * np.repeat(got["ks"][to].copy().view(np.float16).astype(np.float64), 32, -1) * (1 + 2.0 ** -20)
    assert (np.abs(k1[to] - y) <= allowed)[turn != 0].all()


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("layout,n_rot", [(HALF, 128), (PAIRS, 128), (HALF, 40), (PAIRS, 40), (HALF, 8), (HALF, 64), (PAIRS, 96)])
@pytest.mark.parametrize("way", ["still", "down", "apart"])
def test_turned_keys(way, layout, n_rot, k_type, v_type):
    r = np.random.default_rng(n_rot)
    page, H, n = 32, 2, 101
    pool, rows = _filled(r, 8, page, H, k_type, v_type)
    frm, to = (np.arange(n) + 3,) * 2 if way == "still" else _moves(r, way, 8 * page, n)
    turn = r.integers(-5000, 5000, n)
    turn[::5], turn[1::7] = 0, -517
    kvq.kvq_paged_move(pool, i32(frm), i32(to), rope=kvq.Rope(n_rot, layout=layout, amplitude=7.0, device=dev()), turn=i32(turn), staged=way == "down")
    got = _by_slot(pool)
    for name, a in rows.items():     # V moves as it is, and so does what does not turn; other slots stay
        want = a.copy()
        want[to] = a[frm]
        still = np.ones(a.shape, bool)
        if name in ("kq", "k16", "ks"):
            blocks = -(-n_rot // 32)
            part = slice(0, n_rot) if name == "k16" else slice(0, 32 * blocks) if name == "kq" else slice(0, blocks)
            still[to[turn != 0], :, part] = False
        assert np.array_equal(got[name][still], want[still]), name
    k0, k1 = values(rows, v_type)[0], values(got, v_type)[0]
    y, size = rotated(k0[frm], turn, rates(n_rot)[0], 1.0, layout)
    allowed = fp16_bound(y, size)
    if k_type == I8:     # half a step of the new codes
        step = np.repeat(got["ks"][to].copy().view(np.float16).astype(np.float64), 32, -1)
        allowed = allowed + 0.5 * step * (1 + 2.0 ** -20)
    moved = turn != 0
    assert (np.abs(k1[to] - y) <= allowed)[moved].all()


@pytest.mark.parametrize("k_type,v_type", [(I8, Q4), (I8, Q8), (F16, Q4), (F16, Q8)])
@pytest.mark.parametrize("layout,n_rot", [(HALF, 128), (PAIRS, 64), (HALF, 40), (HALF, 0)])
@pytest.mark.parametrize("kind", ["down", "mixed", "reversed"])
def test_staged_moves_of_all_sizes(kind, layout, n_rot, k_type, v_type):
    """Slots that are one another's source, whatever holds the rows meanwhile: the bits of two moves by way of other pages."""
    r = np.random.default_rng(n_rot)
    page, H, half = 64, 3, 13 * 64
    pool, _ = _filled(r, 2 * half // page, page, H, k_type, v_type)
    cut = pool.data.numel() // 2
    start, rope = pool.data.clone(), kvq.Rope(n_rot, layout=layout, device=dev())
    for n in (2, 31, 32, 33, 64, 65, 128, 129, 255, 256, 257, 700):
        frm, to = (x.copy() for x in _moves(r, kind, half, n))
        frm[::9], to[4::11] = -1, 2 ** 30                     # tokens without a slot
        turn = i32(r.integers(-3, 3, n) * 1000)
        there = np.where((frm >= 0) & (to < 2 ** 30), half + np.arange(n), -1)
        pool.data.copy_(start)
        kvq.kvq_paged_move(pool, i32(frm), i32(there), rope=rope, turn=turn, staged=False)
        kvq.kvq_paged_move(pool, i32(there), i32(to), staged=False)
        want = pool.data[:cut].clone()
        pool.data.copy_(start)
        kvq.kvq_paged_move(pool, i32(frm), i32(to), rope=rope, turn=turn, staged=True)
        assert torch.equal(pool.data[:cut], want) and torch.equal(pool.data[cut:], start[cut:]), n


def test_moved_past_32_bits():
    H, page = 8, 256
    n_pages = (5 << 30) // (H * 16 * 4352)
    pool, rope = kvq.PagePool(n_pages, page, H, Q8), kvq.Rope(128, device=dev())
    r = np.random.default_rng(10)
    n = 300
    x = to_dev(_tokens(r, n, 1, H))
    far, near = (n_pages - 3) * page + 7 + np.arange(n), 5 + np.arange(n)
    one, turn = kvq.PagePool(6, page, H, Q8), i32(r.integers(-9, 9, n))
    kvq.kvq_paged_append(one, x[:, 1:1 + H].contiguous(), x[:, 1 + H:].contiguous(), i32(near))
    kvq.kvq_paged_move(one, i32(near), i32(near), rope=rope, turn=turn, staged=False)
    want = [torch.zeros((n, H, 128), device=dev()) for _ in range(2)]
    kvq.kvq_paged_gather(one, i32(near), *want)
    for m, staged in ((n, True), (200, True), (n, False)):
        kvq.kvq_paged_append(pool, x[:, 1:1 + H].contiguous(), x[:, 1 + H:].contiguous(), i32(far))
        got = [torch.zeros((n, H, 128), device=dev()) for _ in range(2)]
        kvq.kvq_paged_move(pool, i32(far[:m]), i32(near[:m]), rope=rope, turn=turn[:m], staged=staged)
        kvq.kvq_paged_move(pool, i32(near[:m]), i32(far[:m]), staged=staged)
        kvq.kvq_paged_gather(pool, i32(far), *got)
        assert torch.equal(got[0][:m], want[0][:m]) and torch.equal(got[1][:m], want[1][:m]) and want[0].any()


def test_a_turn_and_back():
    """Turning keys away and back costs two quantizations, no more."""
    r = np.random.default_rng(9)
    pool, rows = _filled(r, 6, 16, 2, I8, Q8, big=False)
    slots, rope = i32(np.arange(96)), kvq.Rope(128, device=dev())
    for t in (-777, 777):
        kvq.kvq_paged_move(pool, slots, slots, rope=rope, turn=i32(np.full(96, t)), staged=False)
    k0, k1 = values(rows, Q8)[0], values(_by_slot(pool), Q8)[0]
    top = np.abs(k0).max(-1, keepdims=True) * np.sqrt(2)
    # a step is at most sqrt(2) max / 127; the first rounding's error comes back turned (sqrt(2) of it at most), and the second's on top
    assert (np.abs(k1 - k0) <= (1 + np.sqrt(2)) * 0.5 * np.sqrt(2) * top / 127 + 4 * 2.0 ** -11 * top).all()


# ------------------------------------------- streams, graphs and the whole --
def test_a_workspace_of_its_own_on_other_streams():
    """Calls made on a side stream get a workspace that no queued work holds (as kvq_paged_attn)."""
    r = np.random.default_rng(2)
    pool, rows = _filled(r, 40, 64, 8, I8, Q8)
    n = 2000
    side = torch.cuda.Stream()
    frm, to = np.arange(n) + 9, np.arange(n)
    call = kvq.PagedMoveCall(pool, i32(frm), i32(to))
    x = torch.zeros_like(call._own)
    torch.cuda.synchronize()
    at = call._own.data_ptr()
    torch.cuda._sleep(20_000_000)
    del call
    y = torch.full_like(x, 5)          # the freed block, in use by queued work of this stream
    assert y.data_ptr() == at, "the allocator gave other memory: the test shows nothing"
    z = y.clone()
    del y
    f, t = i32(frm), i32(to)
    kvq.kvq_paged_move(pool, f, t, stream=side)
    torch.cuda.synchronize()
    got = _by_slot(pool)
    for name, a in rows.items():
        want = a.copy()
        want[to] = a[frm]
        assert np.array_equal(got[name], want), name
    assert (z == 5).all()


def test_another_current_device_or_a_missing_one_is_refused():
    s = i32([0])
    call = kvq.PagePositionsCall(i32([0, 1]), s, s.clone())
    call._index = 1
    with pytest.raises(ValueError, match="the current device is"):
        call()


@pytest.mark.parametrize("norm", [True, False])
def test_beams(norm):
    """A beam search as a server runs it, its step captured once and replayed: fork, copies in both layers, tables, positions, then
    for each layer the new tokens in and attention.  Against each beam's own history in 64 bits."""
    r = np.random.default_rng(11)
    B, page, H, Hq, layers, most, n_pages, prompt = 6, 16, 2, 6, 2, 5, 40, 21
    rope = kvq.Rope(128, device=dev())
    w = to_dev((1 + 0.2 * r.standard_normal((2, 128))).astype(np.float32)) if norm else [None, None]
    pools = [kvq.PagePool(n_pages, page, H, Q4 if i else Q8) for i in range(layers)]
    for p in pools:
        p.data.fill_(POISON)
    tabs = [torch.full((B, most), -1, dtype=torch.int32, device=dev()) for _ in range(2)]
    lens, free, n_free = i32(np.zeros(B)), i32(r.permutation(n_pages)), i32([n_pages])
    n_new, parent, q_start, status = i32(np.zeros(B)), i32(np.arange(B)), i32(np.zeros(B + 1)), i32(np.zeros(B))
    cf, ct, ch, fs = (i32(np.zeros(B)) for _ in range(4))
    cap = 2 * prompt
    slots, pos = i32(np.zeros(cap)), i32(np.zeros(cap))
    x = torch.zeros((layers, cap, Hq + 2 * H, 128), dtype=torch.float16, device=dev())
    qo = torch.zeros((layers, cap, Hq, 128), dtype=torch.float16, device=dev())
    out, lse = torch.zeros((layers, cap, Hq, 128), device=dev()), torch.zeros((layers, cap, Hq), device=dev())
    calls = [kvq.PageForkCall(page, n_pages, lens, tabs[0], free, n_free, tabs[1], lens, n_free, cf, ct, ch, fs, parent=parent),
             kvq.PageCopyCall(pools, cf, ct, held=ch)]
    back = kvq.PageForkCall(page, n_pages, lens, tabs[1], free, n_free, tabs[0], lens, n_free, cf, ct, ch, fs)
    calls += [back, kvq.PageTablesCall(page, n_pages, lens, n_new, free, n_free, tabs[0], lens, n_free, q_start, slots, status),
              kvq.PagePositionsCall(q_start, lens, pos)]
    for i in range(layers):
        calls += [kvq.QkvCall(x[i, :, :Hq], x[i, :, Hq:Hq + H], x[i, :, Hq + H:], pos, rope, qo[i], pool=pools[i], slots=slots, q_norm=w[0], k_norm=w[1]),
                  kvq.PagedAttnCall(pools[i], qo[i], q_start, cap, lens, tabs[0], True, SM_SCALE, out[i], lse[i])]

    def step():
        for c in calls:
            c()

    step()                     # outside capture first (nothing to add: no place has tokens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = [[np.zeros((2, 0, H, 128), np.float16) for _ in range(B)] for _ in range(layers)]
    copies = 0
    for t in range(20):
        if t == 0:             # two prompts, one place each
            new, par = [prompt, 0, 0, prompt, 0, 0], list(range(B))
        elif t == 1:
            new, par = [1] * B, [0, 0, 0, 3, 3, 3]
        elif t == 12:          # a search ends, the other takes a new start
            new, par = [1, 1, 1, 0, 0, 0], [2, 0, 2, -1, -1, -1]
        elif t == 13:
            new, par = [1, 1, 1, prompt, 0, 0], [0, 1, 2, 3, 4, 5]
        elif t < 12:
            new, par = [1] * B, [int(b // 3 * 3 + r.integers(0, 3)) for b in range(B)]
        else:
            new, par = [1, 1, 1, 1, 0, 0], [int(r.integers(0, 3)) for _ in range(3)] + [3, 4, 5]
        T = sum(new)
        x[:, :T] = to_dev(r.standard_normal((layers, T, Hq + 2 * H, 128)).astype(np.float16))
        n_new.copy_(i32(new))
        parent.copy_(i32(par))
        out.fill_(777)
        graph.replay()
        torch.cuda.synchronize()
        assert not status.any() and not fs.any()
        copies += t > 1
        hist = [[h[p] if p >= 0 else h[0][:, :0] for p in par] for h in hist]
        at = np.concatenate([np.arange(n) + hist[0][b].shape[1] for b, n in enumerate(new)])
        for i in range(layers):
            ka = torch.zeros((T, H, 128), dtype=torch.float16, device=dev())
            kvq.kvq_qkv(None, x[i, :T, Hq:Hq + H], None, i32(at), rope, None, k_out=ka, k_norm=w[1])
            ka, va = ka.cpu().numpy(), x[i, :T, Hq + H:].cpu().numpy()
            t0 = 0
            for b, n in enumerate(new):
                hist[i][b] = np.concatenate([hist[i][b], np.stack([ka[t0:t0 + n], va[t0:t0 + n]])], 1)
                if n:
                    ref = oracle.decode_seq(oracle.quantize_kv(hist[i][b][0], hist[i][b][1], pools[i].v_type), qo[i, t0:t0 + n].cpu().numpy(),
                                            oracle.default_head_map(Hq, H), True, SM_SCALE, pools[i].v_type)
                    assert np.abs(f64(out[i, t0:t0 + n]) - ref["out"]).max() <= 2e-3 and np.abs(f64(lse[i, t0:t0 + n]) - ref["lse"]).max() <= 1e-4, (t, i, b)
                t0 += n
            assert (out[i, T:] == 777).all()
        assert lens.tolist() == [h.shape[1] for h in hist[0]]
        listed = {int(p) for b in range(B) for p in tabs[0][b, :-(-int(lens[b]) // page)]}
        left = free[:int(n_free)].tolist()
        assert len(listed) + len(left) == n_pages and listed | set(left) == set(range(n_pages)), "pages lost or listed twice"
    assert kvq.kvq_wait_timeouts() == 0


@pytest.mark.parametrize("whole_pages", [False, True])
def test_a_context_lets_go_of_its_middle(whole_pages):
    """Tokens dropped, the rest moved (or left in its pages) and its keys turned back: attention as over the shorter context,
    whose keys were written at their new positions, to what one more quantization of K makes."""
    r = np.random.default_rng(12)
    page, H, Hq, L, sink, n_pages = 16, 2, 4, 203, 16, 14
    gap = 48 if whole_pages else 37
    rope, f = kvq.Rope(128, device=dev()), rates(128)[0]
    raw = r.standard_normal((2, L, H, 128)).astype(np.float16)
    pool = kvq.PagePool(n_pages, page, H, Q8)
    table = r.permutation(n_pages)[:-(-L // page)].astype(np.int32)
    slots = table[np.arange(L) // page] * page + np.arange(L) % page
    kvq.kvq_qkv(None, to_dev(raw[0]), to_dev(raw[1]), i32(np.arange(L)), rope, None, pool=pool, slots=i32(slots))
    kept = np.concatenate([np.arange(sink), np.arange(sink + gap, L)])
    n = L - gap
    rest = i32(np.full(n - sink, -gap))
    if whole_pages:
        table = np.concatenate([table[:1], table[1 + gap // page:]])
        kvq.kvq_paged_move(pool, i32(slots[sink + gap:]), i32(slots[sink + gap:]), rope=rope, turn=rest, staged=False)
    else:
        kvq.kvq_paged_move(pool, i32(slots[sink + gap:]), i32(slots[sink:n]), rope=rope, turn=rest)
    tab = i32(np.concatenate([table, np.full(14 - len(table), -1)])[None])
    q = r.standard_normal((1, Hq, 128)).astype(np.float16)
    qo, out, lse = to_dev(q), torch.zeros((1, Hq, 128), device=dev()), torch.zeros((1, Hq), device=dev())
    kvq.kvq_qkv(qo, None, None, i32([n - 1]), rope, qo)
    kvq.kvq_paged_attn(pool, qo, i32([0, 1]), 1, i32([n]), tab, True, SM_SCALE, out, lse)
    k = rotated(raw[0][kept].astype(np.float64), np.arange(n), f, 1.0, HALF)[0]
    v = values(oracle.quantize_kv(raw[1][kept], raw[1][kept], Q8), Q8)[1]
    qv = values(oracle.quantize_kv(qo.cpu().numpy(), qo.cpu().numpy(), Q8), Q8)[0][:, 0]
    # a key is off by half a step (its block's largest value over 127, times sqrt(2) after a turn) twice at most, the first error turned
    step = np.sqrt(2) * np.abs(k).max() * 1.01 / 127
    off = (1 + np.sqrt(2)) * 0.5 * step + 4 * 2.0 ** -11 * np.abs(k).max()
    for h in range(Hq):
        s = k[:, h // 2] @ qv[h] * SM_SCALE
        p = np.exp(s - s.max())
        es = np.abs(qv[h]).sum() * off * SM_SCALE       # of every score
        assert abs(float(lse[0, h]) - (s.max() + np.log(p.sum()))) <= es + 1e-4
        ref = p @ v[h // 2] / p.sum()
        assert (np.abs(f64(out[0, h]) - ref) <= np.abs(v).max() * (np.exp(2 * es) - 1) + 2e-3).all()
        # and nearer than that on the average: with the wrong positions the scores would be other ones
        assert np.corrcoef(f64(out[0, h]), ref)[0, 1] > 0.99


def test_the_fp32_allowance_is_small():
    """What the bounds allow for fp32 arithmetic stays far below fp16's own rounding."""
    assert FP32 < 2.0 ** -19
