"""The paged cache's C ABI and binding without a GPU: exports, the tile record's
layout, and every refusal of a bad argument before the device is touched."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from quantized_kv_cache_03_gb300 import build as B
from quantized_kv_cache_03_gb300 import kvq

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kvq_paged.h")
P = ctypes.c_void_p
BAD, UNSUP = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return kvq.load()


def test_header_and_binding_agree(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(kvq_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(kvq.EXPORTED_PAGED)
    for n in names:
        assert hasattr(lib, n), n


def _pages(**over):
    a = dict(n_pages=10, page_tokens=16, n_kv_heads=2, head_dim=128, k_type=0, v_type=0, data=0x10000)
    a.update(over)
    return kvq.KvqPages(a["n_pages"], a["page_tokens"], a["n_kv_heads"], a["head_dim"], a["k_type"], a["v_type"], a["data"])


BAD_POOLS = [(dict(n_pages=-1), BAD), (dict(page_tokens=0), BAD), (dict(page_tokens=24), BAD), (dict(page_tokens=8), BAD),
             (dict(page_tokens=512), BAD), (dict(n_kv_heads=0), BAD), (dict(n_kv_heads=257), BAD), (dict(head_dim=64), UNSUP),
             (dict(head_dim=100), BAD), (dict(k_type=2), BAD), (dict(v_type=-1), BAD), (dict(n_pages=1 << 28), BAD)]


def test_page_bytes(lib):
    n = ctypes.c_size_t()
    for k, v, tile in ((0, 0, 2048 + 128 + 1024 + 128), (0, 1, 2048 + 128 + 2048 + 128), (1, 0, 4096 + 1024 + 128),
                       (1, 1, 4096 + 2048 + 128)):
        for page in (16, 32, 64, 128, 256):
            p = _pages(page_tokens=page, k_type=k, v_type=v, n_kv_heads=3)
            assert lib.kvq_page_bytes(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value == 3 * (page // 16) * tile
    for over, st in BAD_POOLS:
        p = _pages(**over)
        assert lib.kvq_page_bytes(ctypes.byref(p), ctypes.byref(n)) == st, over
    assert lib.kvq_page_bytes(None, ctypes.byref(n)) == BAD
    assert lib.kvq_page_bytes(ctypes.byref(_pages()), None) == BAD


def _tables(lib, **over):
    a = dict(n_seqs=4, page=16, n_pages=100, lens=0x1000, n_new=0x2000, free=0x3000, n_free=0x4000, table=0x5000, stride=8,
             blocks=8, lens_out=0x6000, n_free_out=0x7000, q_start=0x8000, slots=0x9000, n_tokens=64, status=0xa000)
    a.update(over)
    return lib.kvq_page_tables(a["n_seqs"], a["page"], a["n_pages"], P(a["lens"]), P(a["n_new"]), P(a["free"]), P(a["n_free"]),
                               P(a["table"]), a["stride"], a["blocks"], P(a["lens_out"]), P(a["n_free_out"]), P(a["q_start"]),
                               P(a["slots"]), a["n_tokens"], P(a["status"]), None)


@pytest.mark.parametrize("over", [dict(n_seqs=-1), dict(n_seqs=4097), dict(page=20), dict(n_pages=-1), dict(n_pages=1 << 28),
                                  dict(n_tokens=-1), dict(stride=7), dict(blocks=-1), dict(blocks=1 << 27, stride=1 << 27), dict(lens=0),
                                  dict(n_new=0), dict(free=0), dict(n_free=0), dict(table=0), dict(lens_out=0), dict(n_free_out=0),
                                  dict(q_start=0), dict(slots=0), dict(status=0), dict(lens=0x1002), dict(slots=0x9001)])
def test_tables_refuses(lib, over):
    assert _tables(lib, **over) == BAD


def test_append_and_gather_refuse(lib):
    def append(p=None, k=0x20000, v=0x30000, stride=256, slots=0x40000, n=8, **over):
        return lib.kvq_paged_append(ctypes.byref(_pages(**over)) if p is None else p, P(k), P(v), stride, P(slots), n, None)

    def gather(k=0x20000, v=0x30000, slots=0x40000, n=8, ot=0, **over):
        return lib.kvq_paged_gather(ctypes.byref(_pages(**over)), P(slots), n, ot, P(k), P(v), None)

    for over, st in BAD_POOLS + [(dict(data=0), BAD), (dict(data=0x10040), BAD)]:
        assert append(**over) == st and gather(**over) == st, over
    for kw in (dict(k=0), dict(v=0), dict(k=0x20008), dict(v=0x30002), dict(slots=0), dict(slots=0x40001), dict(n=-1),
               dict(stride=255), dict(stride=250), dict(stride=260), dict(n=1 << 30)):
        assert append(**kw) == BAD, kw
    for kw in (dict(k=0), dict(v=0), dict(k=0x20008), dict(slots=0), dict(n=-1), dict(ot=2), dict(ot=-1)):
        assert gather(**kw) == BAD, kw
    assert append(n=0) == 0 and gather(n=0) == 0 and append(n_pages=0, data=0) == 0


def _attn(lib, size_only=False, ws=0, wsb=0, pool=None, **over):
    a = dict(q=0x20000, q_stride=512, heads=4, tokens=8, seqs=2, max_q=4, q_start=0x30000, lens=0x40000, table=0x50000, ts=8,
             blocks=8, causal=1, hm=None, scale=0.1, ot=0, out=0x60000, lse=0x70000)
    a.update(over)
    hm = None if a["hm"] is None else (ctypes.c_int32 * len(a["hm"]))(*a["hm"])
    pg = _pages(**(pool or {}))
    d = kvq.KvqPagedDesc(ctypes.pointer(pg), a["q"], a["q_stride"], a["heads"], a["tokens"], a["seqs"], a["max_q"], a["q_start"],
                         a["lens"], a["table"], a["ts"], a["blocks"], a["causal"],
                         None if hm is None else ctypes.cast(hm, ctypes.POINTER(ctypes.c_int32)), a["scale"], a["ot"], a["out"], a["lse"])
    if size_only:
        n = ctypes.c_size_t()
        return lib.kvq_paged_attn_workspace_size(ctypes.byref(d), ctypes.byref(n)), n.value
    return lib.kvq_paged_attn(ctypes.byref(d), P(ws), wsb, None)


SHAPES = [dict(heads=0), dict(heads=257), dict(heads=3), dict(tokens=-1), dict(seqs=-1), dict(seqs=4097), dict(max_q=0),
          dict(max_q=9), dict(max_q=(1 << 26) + 1, tokens=(1 << 26) + 1), dict(ts=7), dict(blocks=-1), dict(blocks=1 << 27, ts=1 << 27), dict(scale=float("nan")),
          dict(scale=float("inf")), dict(ot=2), dict(hm=[0, 1, 2, 0]), dict(hm=[0, -1, 0, 0]), dict(tokens=1 << 29)]


@pytest.mark.parametrize("over", SHAPES)
def test_attention_refuses_shapes(lib, over):
    assert _attn(lib, **over) == BAD
    assert _attn(lib, size_only=True, **over)[0] == BAD


@pytest.mark.parametrize("over", [dict(q=0), dict(q=0x20008), dict(q_stride=511), dict(q_stride=504), dict(q_start=0), dict(lens=0),
                                  dict(table=0), dict(out=0), dict(out=0x60008), dict(lse=0x70001), dict(q_start=0x30002)])
def test_attention_refuses_pointers(lib, over):
    assert _attn(lib, **over) == BAD


def test_attention_refuses_pools_and_takes_empty_batches(lib):
    for over, st in BAD_POOLS + [(dict(data=0), BAD)]:
        assert _attn(lib, pool=over) == st, over
    assert lib.kvq_paged_attn(None, None, 0, None) == BAD
    assert _attn(lib, tokens=0) == 0 and _attn(lib, seqs=0) == 0
    assert _attn(lib, size_only=True, tokens=0) == (0, 0)


def test_binding_refuses():
    cpu = torch.device("cpu")
    pool = kvq.PagePool(4, 16, 2, kvq.V_Q4_0, data=torch.zeros(4 * 2 * 3328, dtype=torch.uint8))
    assert pool.page_bytes == 2 * 3328 and pool.device == cpu
    with pytest.raises(ValueError):
        kvq.PagePool(4, 16, 2, kvq.V_Q4_0, data=torch.zeros(5, dtype=torch.uint8))
    with pytest.raises(kvq.KvqError):
        kvq.PagePool(4, 17, 2, kvq.V_Q4_0, data=torch.zeros(5, dtype=torch.uint8))
    k = torch.zeros((3, 2, 128), dtype=torch.float16)
    s = torch.zeros(3, dtype=torch.int32)
    kvq.PagedAppendCall(pool, k, k, s)
    fused = torch.zeros((3, 8, 128), dtype=torch.float16)
    kvq.PagedAppendCall(pool, fused[:, 4:6], fused[:, 6:], s)
    for bad in ((k.float(), k, s), (k, k, s.long()), (k[:2], k, s), (k, fused[:, 6:], s), (k[:, :1], k, s),
                (k.transpose(0, 1), k, s), (torch.zeros((3, 4, 128), dtype=torch.float16)[:, ::2], k, s)):
        with pytest.raises(ValueError):
            kvq.PagedAppendCall(pool, *bad)
    o = torch.zeros((3, 2, 128))
    kvq.PagedGatherCall(pool, s, o, o)
    for bad in ((s, o, o.half()), (s, o.double(), o.double()), (s[:2], o, o)):
        with pytest.raises(ValueError):
            kvq.PagedGatherCall(pool, *bad)
    z = torch.zeros(3, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    tab = torch.zeros((3, 4), dtype=torch.int32)
    q4 = torch.zeros(4, dtype=torch.int32)
    kvq.PageTablesCall(16, 4, z, z, q4, one, tab, z, one, q4, z, z)
    for i, bad in ((0, z.long()), (2, z), (3, z), (4, tab.t()), (4, tab[:2]), (7, z), (8, z.float())):
        args = [z, z, q4, one, tab, z, one, q4, z, z]
        args[i] = bad
        with pytest.raises(ValueError):
            kvq.PageTablesCall(16, 4, *args)
    q = torch.zeros((5, 4, 128), dtype=torch.float16)
    ok = dict(q16=q, q_start=q4, max_q=2, seq_lens=z, block_table=tab, causal=True, sm_scale=0.1, out=torch.zeros((5, 4, 128)),
              lse=torch.zeros((5, 4)), workspace=torch.zeros(8, dtype=torch.uint8))
    kvq.PagedAttnCall(pool, **ok)
    for name, bad in (("q16", q.float()), ("q16", q[0]), ("q_start", z), ("seq_lens", z.long()), ("block_table", tab.t()),
                      ("out", torch.zeros((4, 4, 128))), ("out", q.bfloat16()), ("lse", torch.zeros((5, 3))), ("workspace", z),
                      ("head_map", [0, 1])):
        with pytest.raises(ValueError):
            kvq.PagedAttnCall(pool, **{**ok, name: bad})


def test_tile_record_is_a_bijection():
    """Every byte of a tile belongs to one (position, code) or (position, block)."""
    from paged_cases import scale_index, split_tiles
    si = scale_index()
    assert np.array_equal(np.unique(np.stack([si, si + 1])), np.arange(128))
    u, b = np.meshgrid(np.arange(16), np.arange(4), indexing="ij")
    assert np.array_equal(si, 2 * ((u // 8 * 4 + u % 8 // 2) * 8 + 2 * b + u % 2))   # as the header states it
    for k, v, n in ((0, 0, 3328), (0, 1, 4352), (1, 0, 5248), (1, 1, 6272)):
        rows = split_tiles(np.zeros((2, n), np.uint8), k, v)
        assert sum(a[0].nbytes for a in rows.values()) == n


def test_the_lost_copy_hook_refuses(lib):
    def lose(copy=0, ot=0, pool=None, **over):
        pg = _pages(**(pool or {}))
        d = kvq.KvqPagedDesc(ctypes.pointer(pg), 0x20000, 512, 4, 8, 2, 4, 0x30000, 0x40000, 0x50000, 8, 8, 1, None, 0.1, ot, 0x60000, 0x70000)
        return lib.kvq_debug_paged_lose_copy(ctypes.byref(d), copy, None, 0, None)
    assert lose(copy=-1) == BAD and lose(pool=dict(n_pages=-1)) == BAD
    assert lose(ot=1) == UNSUP and lose(pool=dict(v_type=1)) == UNSUP and lose(pool=dict(k_type=1)) == UNSUP


def test_tensors_of_the_host_are_refused(monkeypatch):
    """Calls over host tensors can be prepared (their checks need no GPU), but not made: no pointer of theirs reaches a kernel."""
    pool = kvq.PagePool(4, 16, 2, kvq.V_Q4_0, data=torch.zeros(4 * 2 * 3328, dtype=torch.uint8))
    k, s, o = torch.zeros((3, 2, 128), dtype=torch.float16), torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2, 128))
    one, q4, tab = torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32)
    attn = kvq.PagedAttnCall(pool, torch.zeros((3, 4, 128), dtype=torch.float16), q4, 1, s, tab, True, 0.1, torch.zeros((3, 4, 128)),
                             workspace=torch.zeros(8, dtype=torch.uint8))
    calls = [kvq.PagedAppendCall(pool, k, k, s), kvq.PagedGatherCall(pool, s, o, o), attn,
             kvq.PageTablesCall(16, 4, s, s, q4, one, tab, s, one, q4, s, s)]
    reached = []
    for c in calls:
        monkeypatch.setattr(c, "_fn", lambda *a: reached.append(a) or 0)
        with pytest.raises(ValueError, match="not on a CUDA device"):
            c()
        with pytest.raises(ValueError, match="not on a CUDA device"):
            c(0)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        kvq.kvq_debug_paged_lose_copy(attn, 0)
    assert not reached


def test_numbers_past_32_bits_are_refused():
    """ctypes cuts an int32 argument off: 2^32 + 16 would arrive as 16.  (Meta tensors have the shapes without the memory.)"""
    def t(*shape, dt=torch.int32):
        return torch.empty(shape, dtype=dt, device="meta")

    big = 2 ** 32
    with pytest.raises(ValueError, match="32 bits"):
        kvq.PagePool(4, big + 16, 2, kvq.V_Q4_0, data=t(4 * 2 * 3328, dt=torch.uint8))
    pool = kvq.PagePool(4, 16, 2, kvq.V_Q4_0, data=t(4 * 2 * 3328, dt=torch.uint8))
    wide = torch.empty_strided((3, 4), (big + 4, 1), dtype=torch.int32, device="meta")
    for page, table, slots in ((big + 16, t(3, 4), t(3)), (16, wide, t(3)), (16, t(3, 4), t(big + 3)), (16, t(3, big + 4), t(3))):
        with pytest.raises(ValueError, match="32 bits"):
            kvq.PageTablesCall(page, 4, t(3), t(3), t(4), t(1), table, t(3), t(1), t(4), slots, t(3))
    kvq.PageTablesCall(16, 4, t(3), t(3), t(4), t(1), t(3, 4), t(3), t(1), t(4), t(3), t(3))
    h = torch.float16
    with pytest.raises(ValueError, match="32 bits"):
        kvq.PagedAppendCall(pool, t(big + 3, 2, 128, dt=h), t(big + 3, 2, 128, dt=h), t(big + 3))
    with pytest.raises(ValueError, match="32 bits"):
        kvq.PagedGatherCall(pool, t(big + 3), t(big + 3, 2, 128, dt=h), t(big + 3, 2, 128, dt=h))
    ok = dict(q16=t(5, 4, 128, dt=h), q_start=t(4), max_q=2, seq_lens=t(3), block_table=t(3, 4), causal=True, sm_scale=0.1,
              out=t(5, 4, 128, dt=h), workspace=t(8, dt=torch.uint8))
    kvq.PagedAttnCall(pool, **ok)
    for over in (dict(max_q=big + 2), dict(block_table=wide), dict(head_map=[0, big, 1, 1]),
                 dict(q16=t(big + 5, 4, 128, dt=h), out=t(big + 5, 4, 128, dt=h))):
        with pytest.raises(ValueError, match="32 bits"):
            kvq.PagedAttnCall(pool, **{**ok, **over})


def test_the_current_stream_without_torchs_private_call(monkeypatch):
    """The binding imports and finds the stream in a torch that lacks the private name."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("kvq_again", kvq.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: type("S", (), {"cuda_stream": 40 + index})())
    assert again._raw_stream(2) == 42


def test_tables_refuse_as_many_rows_as_row_sums_are_held_to(lib):
    """Sums past 2^31 - 1 stay there, so a batch of that many rows could not tell them from a fit."""
    assert _tables(lib, n_tokens=2 ** 31 - 1) == BAD
