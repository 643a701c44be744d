"""The C ABI and binding of include/kvq_tokens.h without a GPU: exports, the
rates of a rotation, and every refusal before the device is touched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from quantized_kv_cache_03_gb300 import build as B
from quantized_kv_cache_03_gb300 import kvq

from tokens_cases import fork_ref, rates, rotated

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvq_tokens.h")
P = ctypes.c_void_p
OK, BAD, UNSUP = kvq.KVQ_OK, kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED
NO_GPU = not os.path.exists("/dev/nvidia0")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return kvq.load()


def test_header_and_binding_agree(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(kvq_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(kvq.EXPORTED_TOKENS)
    for n in names:
        assert hasattr(lib, n), n


def _turns(lib, n_rot=128, base=1e4, scaling=0, factor=1.0, original=0.0, fast=0.0, slow=0.0, turns=True, amp=True):
    t, a = (ctypes.c_uint64 * 64)(), ctypes.c_float(-1)
    st = lib.kvq_rope_turns(n_rot, base, scaling, factor, original, fast, slow, t if turns else None, ctypes.byref(a) if amp else None)
    return st, np.array(t[:max(0, n_rot) // 2 if n_rot <= 128 else 0], np.uint64), a.value


@pytest.mark.parametrize("n_rot", [0, 8, 40, 64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(base=5e5), dict(scaling=1, factor=4.0), dict(scaling=2, factor=8.0), dict(scaling=1, factor=0.25),
                                dict(scaling=3, factor=8.0, original=4096.0, fast=32.0, slow=1.0), dict(scaling=3, factor=40.0, original=300.0, fast=32.0, slow=1.0),
                                dict(scaling=4, factor=8.0, original=8192.0, fast=4.0, slow=1.0)])
def test_rates(lib, n_rot, kw):
    st, t, amp = _turns(lib, n_rot, **kw)
    f, a = rates(n_rot, **kw)
    assert st == OK and abs(amp - a) <= 2.0 ** -24 * a
    part = f / (2 * math.pi)
    part = part - np.floor(part)
    # a few roundings of 2^-53 in power, division and product (the last pairs' logarithm makes the power's error larger),
    # and half a unit of 2^-64, in which the rate is kept
    assert (np.abs(t.astype(np.float64) / 2.0 ** 64 - part) <= 64 * 2.0 ** -53 * part + 2.0 ** -65).all()


def test_far_positions_keep_their_angle(lib):
    """position * rate in wrapping 64-bit integers is the angle less full turns: against 60-digit arithmetic."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194989")
    _, t, _ = _turns(lib)
    for i in (0, 1, 5, 31, 63):
        rate = Decimal(10000) ** (Decimal(-2 * i) / Decimal(128)) / two_pi
        for pos in (1, 4095, 131071, 2 ** 20 + 7, 2 ** 31 - 1, -1, -4096, -2 ** 31):
            want = rate * pos
            want -= want.to_integral_value(rounding="ROUND_FLOOR")
            got = Decimal((int(t[i]) * pos) % 2 ** 64) / Decimal(2 ** 64)
            off = abs(got - want)
            assert min(off, 1 - off) <= abs(pos) * rate * Decimal(2) ** -48 + Decimal(2) ** -52, (i, pos)


@pytest.mark.parametrize("kw,off", [(dict(), -54), (dict(scaling=1, factor=3.0), -52), (dict(scaling=1, factor=0.25), -50), (dict(scaling=2, factor=8.0), -52),
                                    (dict(scaling=3, factor=40.0, original=300.0, fast=32.0, slow=1.0), -52), (dict(scaling=4, factor=8.0, original=8192.0, fast=4.0, slow=1.0), -52)])
def test_rates_to_what_the_header_says(lib, kw, off):
    """Against 40-digit arithmetic: 2^off of a turn per position, and 2^-65 for the unit in which a rate is kept.  With u = 2^-53, a
    plain rate r = base^-e (up to 1) is off by 0.37 u for its exponent's rounding (r e ln base is 1 / 2.718 at most) and 1.05 u of the
    power, by 0.35 u for 2 pi as a double and by u for the division: 2.77 u / (2 pi) < u / 2.  A blend adds its share, two products
    and a sum, less than 5 u / (2 pi); a factor below 1 multiplies all."""
    from decimal import Decimal as D, getcontext
    getcontext().prec = 40
    two_pi, zero = D("6.28318530717958647692528676655900576839433879875021164194989"), D(0)
    scaling, factor, original, fast, slow = kw.get("scaling", 0), *(D(kw.get(k, 1.0)) for k in ("factor", "original", "fast", "slow"))
    for n_rot, base in ((8, 500000.0), (40, 10000.0), (104, 500000.0), (128, 10000.0), (128, 2.0)):
        _, t, _ = _turns(lib, n_rot, base, **kw)
        b = D(base) * factor ** (D(n_rot) / (n_rot - 2)) if scaling == 2 else D(base)
        if scaling == 3:
            lo, hi = (n_rot * (original / (two_pi * k)).ln() / (2 * b.ln()) for k in (fast, slow))
            lo, hi = max(lo.to_integral_value(rounding="ROUND_FLOOR"), zero), min(hi.to_integral_value(rounding="ROUND_CEILING"), D(n_rot - 1))
        for i in range(n_rot // 2):
            r = b ** (D(-2 * i) / n_rot)
            share = [zero, D(1), zero, (i - lo) / max(hi - lo, D("0.001")) if scaling == 3 else zero, (fast - original * r / two_pi) / (fast - slow) if scaling == 4 else zero][scaling]
            share = min(max(share, zero), D(1))
            want = (r / factor * share + r * (1 - share)) / two_pi
            for pos in (1, 4096, 2 ** 22, 2 ** 31 - 1, -2 ** 31):
                d = (D(int(t[i]) * pos % 2 ** 64) / 2 ** 64 - want * pos) % 1
                d = abs(d)
                assert min(d, 1 - d) <= abs(pos) * (D(2) ** off + D(2) ** -65), (n_rot, base, i, pos)


@pytest.mark.parametrize("kw", [dict(n_rot=-8), dict(n_rot=4), dict(n_rot=136), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(scaling=-1), dict(scaling=5), dict(scaling=1, factor=0.0), dict(scaling=2, factor=float("inf")),
                                dict(scaling=3, factor=2.0, original=0.0, fast=32.0, slow=1.0), dict(scaling=4, factor=2.0, original=10.0, fast=1.0, slow=1.0),
                                dict(scaling=4, factor=2.0, original=10.0, fast=4.0, slow=0.0), dict(scaling=3, factor=2.0, original=10.0, fast=float("nan"), slow=1.0),
                                dict(turns=False), dict(amp=False), dict(scaling=2, factor=1e300, n_rot=8)])
def test_rates_refuse(lib, kw):
    assert _turns(lib, **kw)[0] == BAD


def _pages(**over):
    a = dict(n_pages=10, page_tokens=16, n_kv_heads=2, head_dim=128, k_type=0, v_type=0, data=0x10000)
    a.update(over)
    return kvq.KvqPages(a["n_pages"], a["page_tokens"], a["n_kv_heads"], a["head_dim"], a["k_type"], a["v_type"], a["data"])


BAD_POOLS = [(dict(n_pages=-1), BAD), (dict(page_tokens=24), BAD), (dict(n_kv_heads=257), BAD), (dict(head_dim=64), UNSUP), (dict(k_type=2), BAD),
             (dict(n_pages=1 << 28), BAD), (dict(data=0), BAD), (dict(data=0x10040), BAD)]
BAD_ROPES = [dict(n_rot=-8), dict(n_rot=12), dict(n_rot=136), dict(layout=2), dict(layout=-1), dict(amplitude=float("nan")), dict(turns=0), dict(turns=0x9004)]


def _rope(turns=0x9000, n_rot=128, layout=0, amplitude=1.0):
    return kvq.KvqRope(turns, n_rot, layout, amplitude)


def _qkv(lib, pool=None, rope=None, **over):
    """A call on made-up addresses: only what the checks refuse may be asked here."""
    a = dict(q=0x20000, k=0x30000, v=0x40000, qs=512, ks=256, vs=256, n=8, hq=4, hk=2, eps=1e-6, qn=0x50000, kn=0x50200, pos=0x60000,
             qo=0x70000, qos=512, slots=0x80000, ko=0, kos=0, pages=True)
    a.update(over)
    pg, rp = _pages(**(pool or {})), _rope(**(rope or {}))
    d = kvq.KvqQkvDesc(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["n"], a["hq"], a["hk"], a["eps"], a["qn"], a["kn"],
                       ctypes.pointer(rp), a["pos"], a["qo"], a["qos"], ctypes.pointer(pg) if a["pages"] else None, a["slots"], a["ko"], a["kos"])
    return lib.kvq_qkv(ctypes.byref(d), None)


PLAIN = dict(pages=False, ko=0x90000, kos=256, v=0)


@pytest.mark.parametrize("over", [dict(n=-1), dict(hq=-1), dict(hq=257), dict(hk=257, ks=1 << 16, vs=1 << 16), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                  dict(q=0), dict(k=0), dict(v=0), dict(q=0x20008), dict(k=0x30002), dict(v=0x40008), dict(qs=504), dict(qs=516), dict(ks=248),
                                  dict(vs=252), dict(qn=0x50004), dict(kn=0x50008), dict(pos=0), dict(pos=0x60002), dict(qo=0), dict(qo=0x70008), dict(qos=500),
                                  dict(slots=0), dict(slots=0x80001), dict(ko=0x90000, kos=256), dict(pages=False), dict(hk=3, ks=384, vs=384), dict(hk=0),
                                  dict(n=1 << 28), dict(PLAIN, ko=0x90008), dict(PLAIN, kos=248), dict(PLAIN, hk=0), dict(PLAIN, slots=0x80002), dict(qo=0x20000, qos=520), dict(PLAIN, ko=0x30000, kos=264)])
def test_qkv_refuses(lib, over):
    assert _qkv(lib, **over) == BAD


def test_qkv_refuses_pools_and_rotations_and_takes_nothing(lib):
    for over, st in BAD_POOLS:
        assert _qkv(lib, pool=over) == st, over
    for over in BAD_ROPES:
        assert _qkv(lib, rope=over) == BAD, over
    assert lib.kvq_qkv(None, None) == BAD
    assert _qkv(lib, n=0, q=0, k=0, v=0, slots=0, qo=0, pos=0) == OK
    assert _qkv(lib, hq=0, hk=0, pages=False, q=0, k=0) == OK


def _fork(lib, **over):
    a = dict(n=4, page=16, pages=100, lens=0x1000, parent=0x2000, keep=0x3000, table=0x4000, stride=8, most=8, out=0x5000, ostride=8, lens_out=0x6000,
             free=0x7000, n_free=0x8000, n_free_out=0x9000, frm=0xa000, to=0xb000, held=0xc000, status=0xd000, ws=0x10000, wsb=1 << 20)
    a.update(over)
    return lib.kvq_page_fork(a["n"], a["page"], a["pages"], P(a["lens"]), P(a["parent"]), P(a["keep"]), P(a["table"]), a["stride"], a["most"],
                             P(a["out"]), a["ostride"], P(a["lens_out"]), P(a["free"]), P(a["n_free"]), P(a["n_free_out"]), P(a["frm"]), P(a["to"]),
                             P(a["held"]), P(a["status"]), P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("over", [dict(n=-1), dict(n=4097), dict(page=20), dict(pages=-1), dict(pages=1 << 28), dict(stride=7), dict(ostride=7), dict(most=-1),
                                  dict(most=1 << 27, stride=1 << 27, ostride=1 << 27), dict(lens=0), dict(lens=0x1002), dict(parent=0x2001), dict(keep=0x3002),
                                  dict(table=0), dict(out=0), dict(lens_out=0), dict(free=0), dict(n_free=0), dict(n_free_out=0), dict(frm=0), dict(to=0),
                                  dict(held=0), dict(status=0), dict(out=0x4000), dict(out=0x4000, parent=0, ostride=9)])
def test_fork_refuses(lib, over):
    assert _fork(lib, **over) == BAD


def test_fork_workspace(lib):
    n = ctypes.c_size_t()
    for args in ((-1, 5), (4097, 5), (3, -1)):
        assert lib.kvq_page_fork_workspace_size(*args, ctypes.byref(n)) == BAD
    assert lib.kvq_page_fork_workspace_size(3, 5, None) == BAD
    assert lib.kvq_page_fork_workspace_size(4096, 1 << 27, ctypes.byref(n)) == OK and n.value >= 7 << 27
    if not NO_GPU:
        assert _fork(lib, wsb=16) == kvq.KVQ_ERR_WORKSPACE


def _copy(lib, pools=None, n_pools=None, frm=0x20000, to=0x30000, held=0x40000, n=5):
    pools = [_pages(**over) for over in (pools if pools is not None else [{}, dict(data=0x50000)])]
    arr = (kvq.KvqPages * max(1, len(pools)))(*pools)
    return lib.kvq_page_copy(arr, len(pools) if n_pools is None else n_pools, P(frm), P(to), P(held), n, None)


def test_copy_refuses(lib):
    for over, st in BAD_POOLS:
        assert _copy(lib, [over]) == st, over
    for other in (dict(n_pages=11), dict(page_tokens=32)):
        assert _copy(lib, [{}, other]) == BAD, other
    for kw in (dict(n=-1), dict(n_pools=-1), dict(n_pools=129), dict(frm=0), dict(to=0), dict(frm=0x20002), dict(held=0x40001), dict(n=1 << 29)):
        assert _copy(lib, **kw) == BAD, kw
    assert lib.kvq_page_copy(None, 1, P(0x20000), P(0x30000), None, 5, None) == BAD
    assert _copy(lib, n=0) == OK and _copy(lib, []) == OK and _copy(lib, [dict(n_pages=0, data=0)]) == OK


def _move(lib, pool=None, rope=None, frm=0x20000, to=0x30000, n=5, turn=0x40000, staged=0, ws=0, wsb=0):
    rp = None if rope is None else ctypes.byref(_rope(**rope))
    return lib.kvq_paged_move(ctypes.byref(_pages(**(pool or {}))), P(frm), P(to), n, rp, P(turn), staged, P(ws), wsb, None)


def test_move_refuses(lib):
    n = ctypes.c_size_t()
    for over, st in BAD_POOLS:
        assert _move(lib, pool=over, rope={}) == st, over
    for over in BAD_ROPES:
        assert _move(lib, rope=over) == BAD, over
    for kw in (dict(rope=None), dict(rope={}, turn=0), dict(rope={}, turn=0x40002), dict(rope={}, n=-1), dict(rope={}, n=1 << 30), dict(rope={}, frm=0),
               dict(rope={}, to=0x30001)):
        assert _move(lib, **kw) == BAD, kw
    assert lib.kvq_paged_move(None, P(0x20000), P(0x30000), 5, None, None, 0, None, 0, None) == BAD
    assert _move(lib, rope={}, n=0, frm=0, to=0) == OK and _move(lib, pool=dict(n_pages=0, data=0), turn=0) == OK
    assert lib.kvq_paged_move_workspace_size(ctypes.byref(_pages()), -1, ctypes.byref(n)) == BAD
    assert lib.kvq_paged_move_workspace_size(ctypes.byref(_pages(page_tokens=17)), 1, ctypes.byref(n)) == BAD
    assert lib.kvq_paged_move_workspace_size(ctypes.byref(_pages()), 1, None) == BAD
    for k, v, row in ((0, 0, 208), (0, 1, 272), (1, 0, 336), (1, 1, 400)):
        assert lib.kvq_paged_move_workspace_size(ctypes.byref(_pages(k_type=k, v_type=v)), 7, ctypes.byref(n)) == OK and n.value == 7 * 2 * row


def test_positions_refuse(lib):
    def call(n=3, qs=0x1000, lens=0x2000, t=8, pos=0x3000):
        return lib.kvq_page_positions(n, P(qs), P(lens), t, P(pos), None)
    for kw in (dict(n=-1), dict(n=4097), dict(t=-1), dict(t=2 ** 31 - 1), dict(qs=0), dict(lens=0), dict(pos=0), dict(qs=0x1001), dict(pos=0x3002)):
        assert call(**kw) == BAD, kw
    assert call(t=0, pos=0) == OK


def _pool(n_pages=4, page=16, heads=2):
    return kvq.PagePool(n_pages, page, heads, kvq.V_Q4_0, data=torch.zeros(n_pages * heads * (page // 16) * 3328, dtype=torch.uint8))


def test_binding_refuses():
    h, i = torch.float16, torch.int32
    q, k, s = torch.zeros((3, 4, 128), dtype=h), torch.zeros((3, 2, 128), dtype=h), torch.zeros(3, dtype=i)
    rope, pool, w = kvq.Rope(64, device="cpu"), _pool(), torch.ones(128)
    ok = dict(q16=q, k16=k, v16=k, positions=s, rope=rope, q_out=q, pool=pool, slots=s, q_norm=w, k_norm=w)
    kvq.QkvCall(**ok)
    fused = torch.zeros((3, 8, 128), dtype=h)
    kvq.QkvCall(**{**ok, "q16": fused[:, :4], "k16": fused[:, 4:6], "v16": fused[:, 6:], "q_out": fused[:, :4]})
    kvq.QkvCall(q, k, None, s, rope, q, k_out=k)
    kvq.QkvCall(q, None, None, s, rope, q)
    kvq.QkvCall(None, k, k, s, rope, None, pool=pool, slots=s)
    kvq.QkvCall(q, k, None, None, None, q, k_out=k, q_norm=w, k_norm=w)
    for over in (dict(q16=q.float()), dict(q16=q[:2]), dict(q16=None), dict(k16=k[:, :1]), dict(k16=None), dict(v16=None), dict(v16=q), dict(positions=s.long()),
                 dict(positions=s[:2]), dict(positions=None), dict(q_out=None), dict(q_out=k), dict(q_out=q[:2]), dict(pool=None), dict(slots=None), dict(slots=s[:2]),
                 dict(k_out=k), dict(q_norm=w[:64]), dict(q_norm=w.half()), dict(k_norm=w.double()), dict(q16=q.transpose(0, 1)),
                 dict(pool=_pool(heads=1)), dict(q16=None, q_out=None, k16=None, v16=None, pool=None)):
        with pytest.raises(ValueError):
            kvq.QkvCall(**{**ok, **over})
    with pytest.raises(ValueError):
        kvq.QkvCall(q, k, None, s, rope, q, k_out=q)
    with pytest.raises(ValueError):
        kvq.Rope(64, layout=3, device="cpu")
    with pytest.raises(ValueError):
        kvq.Rope(2 ** 32 + 64, device="cpu")
    for kw in (dict(n_rot=20), dict(n_rot=136), dict(base=0.5), dict(scaling=9), dict(scaling=kvq.ROPE_BY_TURNS, factor=2.0)):
        with pytest.raises(kvq.KvqError):
            kvq.Rope(**kw, device="cpu")
    z, one, tab, free, out = torch.zeros(3, dtype=i), torch.zeros(1, dtype=i), torch.zeros((3, 5), dtype=i), torch.zeros(9, dtype=i), torch.zeros((3, 5), dtype=i)
    args = [16, 9, z, tab, free, one, out, z, one, z, z, z, z]
    kvq.PageForkCall(*args, parent=z, keep=z)
    for at, bad in ((1, 10), (2, z.long()), (3, tab.t()), (3, tab[:2]), (4, one), (5, z), (6, out[:, :4]), (6, out.long()), (7, one), (8, z), (9, z[:2]), (12, None)):
        with pytest.raises(ValueError):
            kvq.PageForkCall(*args[:at], bad, *args[at + 1:])
    for kw in (dict(parent=z.long()), dict(keep=one), dict(workspace=z)):
        with pytest.raises(ValueError):
            kvq.PageForkCall(*args, **kw)
    kvq.PageCopyCall([pool, _pool()], z, z, held=z)
    kvq.PageCopyCall([], z, z)
    for a in (([pool], z.long(), z), ([pool], z, one), ([pool], z, z, one), ([pool] * 129, z, z)):
        with pytest.raises(ValueError):
            kvq.PageCopyCall(*a)
    kvq.PagedMoveCall(pool, z, z, rope=rope, turn=z)
    kvq.PagedMoveCall(pool, z, z, staged=False)
    for kw in (dict(rope=rope), dict(turn=z), dict(rope=rope, turn=one), dict(rope=rope, turn=z.long()), dict(workspace=z)):
        with pytest.raises(ValueError):
            kvq.PagedMoveCall(pool, z, z, **kw)
    with pytest.raises(ValueError):
        kvq.PagedMoveCall(pool, z, one)
    kvq.PagePositionsCall(torch.zeros(4, dtype=i), z, free)
    for a in ((z, z, free), (torch.zeros(4, dtype=i), z.long(), free), (torch.zeros(4, dtype=i), z, tab)):
        with pytest.raises(ValueError):
            kvq.PagePositionsCall(*a)


def test_tensors_of_the_host_are_refused(monkeypatch):
    i = torch.int32
    q, k, s = torch.zeros((3, 4, 128), dtype=torch.float16), torch.zeros((3, 2, 128), dtype=torch.float16), torch.zeros(3, dtype=i)
    one, tab, free = torch.zeros(1, dtype=i), torch.zeros((3, 5), dtype=i), torch.zeros(9, dtype=i)
    pool, rope = _pool(), kvq.Rope(64, device="cpu")
    calls = [kvq.QkvCall(q, k, k, s, rope, q, pool=pool, slots=s), kvq.PageForkCall(16, 9, s, tab, free, one, tab.clone(), s, one, s, s, s, s),
             kvq.PageCopyCall([pool], s, s), kvq.PagedMoveCall(pool, s, s), kvq.PagePositionsCall(torch.zeros(4, dtype=i), s, s)]
    reached = []
    for c in calls:
        monkeypatch.setattr(c, "_fn", lambda *a: reached.append(a) or 0)
        for stream in (None, 0):
            with pytest.raises(ValueError, match="not on a CUDA device"):
                c(stream)
    assert not reached


def test_numbers_past_32_bits_are_refused():
    def t(*shape, dt=torch.int32):
        return torch.empty(shape, dtype=dt, device="meta")

    big = 2 ** 32
    pool = kvq.PagePool(4, 16, 2, kvq.V_Q4_0, data=t(4 * 2 * 3328, dt=torch.uint8))
    q = t(big + 3, 2, 128, dt=torch.float16)
    with pytest.raises(ValueError, match="32 bits"):
        kvq.QkvCall(q, q, q, t(big + 3), None, q, pool=pool, slots=t(big + 3))
    with pytest.raises(ValueError, match="32 bits"):
        kvq.PagePositionsCall(t(4), t(3), t(big + 3))
    with pytest.raises(ValueError, match="32 bits"):
        kvq.PageCopyCall([pool], t(big + 3), t(big + 3))
    with pytest.raises(ValueError, match="32 bits"):
        kvq.PagedMoveCall(pool, t(big + 3), t(big + 3), staged=False)
    z = t(3)
    for page, pages, table in ((big + 16, 4, t(3, 4)), (16, big + 4, t(3, 4)), (16, 4, t(3, big + 4))):
        with pytest.raises(ValueError, match="32 bits"):
            kvq.PageForkCall(page, pages, z, table, t(pages), t(1), table, z, t(1), z, z, z, z, workspace=t(8, dt=torch.uint8))


def test_plain_forms_agree_with_themselves():
    """The references the GPU tests use, on hand-worked cases."""
    x = np.zeros((1, 1, 128))
    x[0, 0, 0], x[0, 0, 64], x[0, 0, 1] = 1, 2, 3
    quarter = np.zeros(64)
    quarter[0] = math.pi / 2
    y, size = rotated(x, [1], quarter, 1.0, kvq.ROPE_HALF)
    assert np.allclose(y[0, 0, [0, 64, 1]], [-2, 1, 3]) and size[0, 0, 0] == 3 and size[0, 0, 1] == 3
    y, _ = rotated(x, [-1], quarter, 2.0, kvq.ROPE_PAIRS)
    assert np.allclose(y[0, 0, [0, 1, 64]], [6, -2, 4])
    # pages of 4: two beams of 6 positions on a shared first page; place 1 goes on with place 0, place 2 keeps 2 of place 0
    table = np.array([[7, 3], [7, 5], [1, -1]], np.int32)
    got = fork_ref(4, 10, [6, 6, 4], table, np.arange(10, 20, dtype=np.int32) % 10, 2, np.full((3, 2), -9, np.int32), 2, [0, 0, 0], [6, 6, 2])
    assert got["table_out"].tolist() == [[7, 3], [7, 5], [1, -9]]      # pages 1 and 5 come back, in order, and are handed out
    assert got["lens"].tolist() == [6, 6, 2] and got["status"].tolist() == [0, 0, 0] and got["n_free"].tolist() == [2]
    assert (got["copy_from"].tolist(), got["copy_to"].tolist(), got["copy_held"].tolist()) == ([-1, 3, 7], [-1, 5, 1], [0, 2, 2])
    assert got["free"].tolist() == [0, 1, 1, 5, 4, 5, 6, 7, 8, 9]
