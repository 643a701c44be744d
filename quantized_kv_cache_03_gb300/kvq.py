"""ctypes binding of libkvq.so (include/kvq.h, and include/kvq_paged.h for the
paged cache): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; torch only
provides device memory and the stream handle.  Importing this module does not
load the library; the first call does, and raises if libkvq.so is missing --
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import threading
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkvq.so")

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_CAPACITY = 3
KVQ_ERR_WORKSPACE = 4
KVQ_ERR_CUDA = 5
KVQ_ERR_TIMEOUT = 6
V_Q4_0 = 0
V_Q8_0 = 1
K_I8 = 0    # K: int8 codes + fp16 scale per 32 (query quantized the same way)
K_F16 = 1   # K: fp16 values (query unquantized)
LAYOUT_TILES = 0   # segment code bytes in 16-token tiles, fragment order
LAYOUT_ROWS = 1    # one row per token in element order
HEAD_DIM = 128
SEG_ALIGN = 64
QBLOCK = 32

EXPORTED = ("kvq_append", "kvq_decode_attn", "kvq_decode_workspace_size", "kvq_decode_attn_multi",
            "kvq_decode_multi_workspace_size", "kvq_decode_attn_noalloc", "kvq_wait_timeouts",
            "kvq_reset_wait_timeouts", "kvq_status_string", "kvq_debug_qk", "kvq_debug_lose_stage",
            "kvq_debug_plan", "kvq_layout_model_default", "kvq_layout_cost", "kvq_choose_layout")
EXPORTED_PAGED = ("kvq_page_bytes", "kvq_page_tables", "kvq_paged_append", "kvq_paged_gather", "kvq_paged_attn",
                  "kvq_paged_attn_workspace_size", "kvq_debug_paged_lose_copy")
OUT_F32 = 0    # type of computed values
OUT_F16 = 1
MAX_PAGED_SEQS = 4096
PAGE_RELEASE = -1
MAX_CALLS = 16
MAX_T_Q = 4096
MAX_T_Q_APPEND = 8
NOALLOC_SCRATCH_BYTES = 32 << 20


class KvqSegment(ctypes.Structure):
    _fields_ = [("k_q", c_void_p), ("k_s", c_void_p), ("v_q", c_void_p), ("v_s", c_void_p),
                ("cap", c_int32), ("len", c_int32), ("pos0", c_int32), ("layout", c_int32)]


class KvqCache(ctypes.Structure):
    _fields_ = [("n_seqs", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("v_type", c_int32), ("max_segs", c_int32), ("n_segs", POINTER(c_int32)),
                ("segs", POINTER(KvqSegment)), ("k_type", c_int32), ("reserved", c_int32)]


class KvqDecodeDesc(ctypes.Structure):
    _fields_ = [("cache", POINTER(KvqCache)), ("q16", c_void_p), ("n_q_heads", c_int32), ("t_q", c_int32),
                ("causal_tail", c_int32), ("seq_lens", c_void_p), ("max_len", c_int32),
                ("head_map", POINTER(c_int32)), ("sm_scale", c_float), ("out", c_void_p), ("lse", c_void_p),
                ("k16_new", c_void_p), ("v16_new", c_void_p)]


class KvqLayoutModel(ctypes.Structure):
    _fields_ = [("us_per_byte", ctypes.c_double), ("us_per_op", ctypes.c_double),
                ("ops_rows_per_tile", ctypes.c_double)]


class KvqPlanLaunch(ctypes.Structure):
    _fields_ = [("kernel", c_int32), ("n_tiles8", c_int32), ("warps", c_int32), ("chunk", c_int32),
                ("chunk0", c_int32), ("n_ctas", c_int32), ("n_rows", c_int32)]


class KvqPages(ctypes.Structure):
    _fields_ = [("n_pages", c_int32), ("page_tokens", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("k_type", c_int32), ("v_type", c_int32), ("data", c_void_p)]


class KvqPagedDesc(ctypes.Structure):
    _fields_ = [("pages", POINTER(KvqPages)), ("q16", c_void_p), ("q_stride", c_int64), ("n_q_heads", c_int32),
                ("n_tokens", c_int32), ("n_seqs", c_int32), ("max_q", c_int32), ("q_start", c_void_p),
                ("seq_lens", c_void_p), ("block_table", c_void_p), ("table_stride", c_int32),
                ("max_blocks", c_int32), ("causal", c_int32), ("head_map", POINTER(c_int32)), ("sm_scale", c_float),
                ("out_type", c_int32), ("out", c_void_p), ("lse", c_void_p)]


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, status_string(status), status))


_lib = None
_lock = threading.Lock()


def load():
    """Load libkvq.so (built by ``__graft_entry__.build()``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libkvq.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
            lib = ctypes.CDLL(LIB_PATH)
            lib.kvq_status_string.restype = ctypes.c_char_p
            lib.kvq_status_string.argtypes = [c_int32]
            lib.kvq_append.restype = c_int32
            lib.kvq_append.argtypes = [POINTER(KvqCache), c_int32, POINTER(c_int32), POINTER(c_int32),
                                       c_void_p, c_void_p, c_void_p]
            lib.kvq_decode_attn.restype = c_int32
            lib.kvq_decode_attn.argtypes = [POINTER(KvqCache), c_void_p, c_int32, c_int32, c_int32, c_void_p,
                                            c_int32, POINTER(c_int32), c_float, c_void_p, c_void_p, c_void_p,
                                            c_size_t, c_void_p]
            lib.kvq_decode_workspace_size.restype = c_int32
            lib.kvq_decode_workspace_size.argtypes = [POINTER(KvqCache), c_int32, c_int32, c_int32,
                                                      POINTER(c_int32), POINTER(c_size_t)]
            lib.kvq_decode_attn_multi.restype = c_int32
            lib.kvq_decode_attn_multi.argtypes = [c_int32, POINTER(KvqDecodeDesc), c_void_p, c_size_t, c_void_p]
            lib.kvq_decode_multi_workspace_size.restype = c_int32
            lib.kvq_decode_multi_workspace_size.argtypes = [c_int32, POINTER(KvqDecodeDesc), POINTER(c_size_t)]
            lib.kvq_decode_attn_noalloc.restype = c_int32
            lib.kvq_decode_attn_noalloc.argtypes = [POINTER(KvqCache), c_void_p, c_int32, c_int32, c_int32,
                                                    c_void_p, c_int32, POINTER(c_int32), c_float, c_void_p,
                                                    c_void_p, c_void_p]
            lib.kvq_wait_timeouts.restype = c_int32
            lib.kvq_wait_timeouts.argtypes = [POINTER(ctypes.c_uint32)]
            lib.kvq_reset_wait_timeouts.restype = c_int32
            lib.kvq_reset_wait_timeouts.argtypes = []
            lib.kvq_layout_model_default.restype = c_int32
            lib.kvq_layout_model_default.argtypes = [POINTER(KvqLayoutModel)]
            lib.kvq_layout_cost.restype = c_int32
            lib.kvq_layout_cost.argtypes = [c_int32, c_int32, c_int32, POINTER(KvqLayoutModel),
                                            POINTER(ctypes.c_double)]
            lib.kvq_choose_layout.restype = c_int32
            lib.kvq_choose_layout.argtypes = [c_int32, c_int32, c_int32, POINTER(KvqLayoutModel), POINTER(c_int32)]
            lib.kvq_debug_lose_stage.restype = c_int32
            lib.kvq_debug_lose_stage.argtypes = lib.kvq_decode_attn.argtypes
            lib.kvq_debug_qk.restype = c_int32
            lib.kvq_debug_qk.argtypes = [POINTER(KvqCache), c_void_p, c_int32, c_int32, c_void_p, c_int32,
                                         POINTER(c_int32), c_void_p, c_void_p, c_void_p, POINTER(c_int32),
                                         c_void_p]
            lib.kvq_debug_plan.restype = c_int32
            lib.kvq_debug_plan.argtypes = [c_int32, POINTER(KvqDecodeDesc), c_int32, POINTER(c_int32),
                                           POINTER(KvqPlanLaunch), c_int32, POINTER(c_int32), POINTER(c_size_t),
                                           POINTER(c_int32)]
            lib.kvq_page_bytes.restype = c_int32
            lib.kvq_page_bytes.argtypes = [POINTER(KvqPages), POINTER(c_size_t)]
            lib.kvq_page_tables.restype = c_int32
            lib.kvq_page_tables.argtypes = [c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                            c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                            c_int32, c_void_p, c_void_p]
            lib.kvq_paged_append.restype = c_int32
            lib.kvq_paged_append.argtypes = [POINTER(KvqPages), c_void_p, c_void_p, c_int64, c_void_p, c_int32,
                                             c_void_p]
            lib.kvq_paged_gather.restype = c_int32
            lib.kvq_paged_gather.argtypes = [POINTER(KvqPages), c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                             c_void_p]
            lib.kvq_paged_attn.restype = c_int32
            lib.kvq_paged_attn.argtypes = [POINTER(KvqPagedDesc), c_void_p, c_size_t, c_void_p]
            lib.kvq_debug_paged_lose_copy.restype = c_int32
            lib.kvq_debug_paged_lose_copy.argtypes = [POINTER(KvqPagedDesc), c_int32, c_void_p, c_size_t, c_void_p]
            lib.kvq_paged_attn_workspace_size.restype = c_int32
            lib.kvq_paged_attn_workspace_size.argtypes = [POINTER(KvqPagedDesc), POINTER(c_size_t)]
            _lib = lib
    return _lib


def status_string(s: int) -> str:
    return load().kvq_status_string(int(s)).decode()


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _i32(vals):
    vals = [int(v) for v in vals]
    return (c_int32 * max(1, len(vals)))(*vals)


class Cache:
    """A batch of append-only segmented caches (device memory from torch).

    Holds the host descriptor of include/kvq.h and keeps the segment tensors
    alive.  Segment arrays are allocated with the byte layout of kvq_segment.
    """

    def __init__(self, n_seqs: int, n_kv_heads: int, v_type: int, max_segs: int = 8,
                 head_dim: int = HEAD_DIM, device=None, k_type: int = K_I8):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.n_seqs, self.n_kv_heads, self.v_type, self.head_dim = n_seqs, n_kv_heads, v_type, head_dim
        self.k_type = k_type
        self.max_segs = max_segs
        self._segs = (KvqSegment * max(1, n_seqs * max_segs))()
        self._nsegs = (c_int32 * max(1, n_seqs))()
        self.desc = KvqCache(n_seqs, n_kv_heads, head_dim, v_type, max_segs,
                             ctypes.cast(self._nsegs, POINTER(c_int32)),
                             ctypes.cast(self._segs, POINTER(KvqSegment)), k_type, 0)
        self.tensors = [[] for _ in range(n_seqs)]

    def seg(self, b: int, k: int) -> KvqSegment:
        return self._segs[b * self.max_segs + k]

    def n_segs(self, b: int) -> int:
        return self._nsegs[b]

    def add_segment(self, b: int, cap: int, layout=LAYOUT_TILES):
        """Open a new segment of `cap` tokens (rounded up to 64) for sequence b,
        its code bytes in `layout` (LAYOUT_TILES, LAYOUT_ROWS, or "auto": the
        layout kvq_choose_layout picks for `cap` expected tokens)."""
        if layout == "auto":
            layout = choose_layout(self.k_type, self.v_type, max(1, int(cap)))
        ns = self._nsegs[b]
        if ns >= self.max_segs:
            raise ValueError("sequence %d already has max_segs segments" % b)
        cap = max(SEG_ALIGN, (int(cap) + SEG_ALIGN - 1) // SEG_ALIGN * SEG_ALIGN)
        H, D = self.n_kv_heads, self.head_dim
        vb = D // 2 if self.v_type == V_Q4_0 else D
        f16k = self.k_type == K_F16
        t = dict(k_q=torch.empty((H, cap, D), dtype=torch.int16 if f16k else torch.int8, device=self.device),
                 k_s=None if f16k else torch.empty((H, cap, D // QBLOCK), dtype=torch.int16, device=self.device),
                 v_q=torch.empty((H, cap, vb), dtype=torch.uint8, device=self.device),
                 v_s=torch.empty((H, cap, D // QBLOCK), dtype=torch.int16, device=self.device))
        pos0 = 0
        if ns:
            prev = self.seg(b, ns - 1)
            pos0 = prev.pos0 + prev.len
        s = self.seg(b, ns)
        s.k_q, s.k_s, s.v_q, s.v_s = (0 if t[n] is None else t[n].data_ptr() for n in ("k_q", "k_s", "v_q", "v_s"))
        s.cap, s.len, s.pos0, s.layout = cap, 0, pos0, int(layout)
        self.tensors[b].append(t)
        self._nsegs[b] = ns + 1
        return t

    def length(self, b: int) -> int:
        ns = self._nsegs[b]
        if not ns:
            return 0
        s = self.seg(b, ns - 1)
        return s.pos0 + s.len

    def lengths(self):
        return [self.length(b) for b in range(self.n_seqs)]

    def export(self, b: int, raw: bool = False):
        """Sequence b copied to host numpy arrays.  raw=False: the filled
        positions, [H][L][row] per array in logical row order.  raw=True: one
        dict per segment with the whole arrays as stored ([H][cap][row], code
        bytes in their in-tile order for tile-layout segments) plus its "len"
        and "layout".  F16 K caches give "k16" (fp16 bits) instead of "kq" and
        "ks"."""
        import numpy as np
        f16k = self.k_type == K_F16
        arrays = ((("k16", "k_q", np.uint16),) if f16k else (("kq", "k_q", np.uint8), ("ks", "k_s", np.uint16))) + \
            (("vq", "v_q", np.uint8), ("vs", "v_s", np.uint16))
        parts = {n: [] for n, _, _ in arrays}
        segs = []
        for k in range(self._nsegs[b]):
            s, t = self.seg(b, k), self.tensors[b][k]
            seg = {"len": s.len, "layout": s.layout}
            for name, key, view in arrays:
                a = t[key].cpu().numpy().view(view)
                seg[name] = a
                if not raw and name in ("kq", "vq", "k16") and s.layout == LAYOUT_TILES:
                    a = untile_codes(a, name, self.v_type)
                parts[name].append(a[:, :s.len])
            segs.append(seg)
        if raw:
            return segs
        return {n: np.concatenate(v, axis=1) for n, v in parts.items()}


def _tile_index(name: str, v_type: int):
    """idx[u, j] = in-tile offset of byte j of the tile's token u (the tile
    layout of include/kvq.h, head_dim 128)."""
    import numpy as np
    u = np.arange(16)[:, None]
    sub, gu, e = u // 8, u % 8, u % 2
    cu = gu // 2
    if name == "k16":   # fp16 elements (offsets in 2-byte units)
        j = np.arange(128)[None, :]
        return ((j // 16) * 512 + (4 * gu + (j % 8) // 2) * 16 + 4 * (sub + 2 * ((j % 16) // 8)) + 2 * (j % 2)) // 2
    if name == "kq":
        j = np.arange(128)[None, :]
        return ((2 * sub + j // 64) * 32 + 4 * gu + (j % 32) // 8) * 16 + 8 * ((j // 32) % 2) + j % 8
    if v_type == V_Q4_0:
        j = np.arange(64)[None, :]
        return (sub * 32 + 4 * ((j % 16) // 2) + cu) * 16 + 4 * (j // 16) + 2 * e + j % 2
    j = np.arange(128)[None, :]
    return (((2 * sub + j // 64) * 32 + 4 * ((j % 32) // 4) + cu) * 16 + 8 * ((j // 32) % 2)
            + 4 * ((j % 4) // 2) + 2 * (j % 2) + e)


def untile_codes(a, name: str, v_type: int):
    """Stored code bytes [H][cap][row] -> logical row order (cap % 16 == 0)."""
    H, cap, row = a.shape
    idx = _tile_index(name, v_type)
    tiles = a.reshape(H, cap // 16, 16 * row)
    return tiles[:, :, idx].reshape(H, cap, row)


def kvq_append(cache: Cache, seq_ids, n_new, k16: torch.Tensor, v16: torch.Tensor, stream=None) -> None:
    """kvq_append of include/kvq.h.  k16/v16: fp16 [sum(n_new)][Hkv][D] on the device."""
    ids, nn = list(seq_ids), list(n_new)
    st = load().kvq_append(ctypes.byref(cache.desc), len(ids), _i32(ids), _i32(nn), _ptr(k16), _ptr(v16),
                           _stream(stream))
    if st:
        raise KvqError(st, "kvq_append")


def kvq_decode_workspace_size(cache: Cache, n_q_heads: int, t_q: int, max_len: int, head_map=None) -> int:
    """Bytes of workspace kvq_decode_attn needs for these arguments."""
    size = c_size_t(0)
    hm = None if head_map is None else _i32(head_map)
    st = load().kvq_decode_workspace_size(ctypes.byref(cache.desc), n_q_heads, t_q, max_len, hm,
                                          ctypes.byref(size))
    if st:
        raise KvqError(st, "kvq_decode_workspace_size")
    return size.value


def kvq_decode_attn(cache: Cache, q16: torch.Tensor, n_q_heads: int, t_q: int, causal_tail: bool,
                    seq_lens: torch.Tensor, max_len: int, head_map, sm_scale: float, out: torch.Tensor,
                    lse: torch.Tensor, workspace: torch.Tensor | None, stream=None) -> None:
    """kvq_decode_attn of include/kvq.h (workspace: a uint8 device tensor of at
    least kvq_decode_workspace_size() bytes, or None when that size is 0)."""
    hm = None if head_map is None else _i32(head_map)
    st = load().kvq_decode_attn(ctypes.byref(cache.desc), _ptr(q16), n_q_heads, t_q, int(causal_tail),
                                _ptr(seq_lens), max_len, hm, float(sm_scale), _ptr(out), _ptr(lse),
                                _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                _stream(stream))
    if st:
        raise KvqError(st, "kvq_decode_attn")


def _descs(calls):
    """calls: sequence of dicts with the per-cache arguments of kvq_decode_attn
    (cache, q16, n_q_heads, t_q, causal_tail, seq_lens, max_len, head_map,
    sm_scale, out, lse) and optionally k16_new / v16_new (fused append);
    tensors may be None for a size query."""
    arr = (KvqDecodeDesc * max(1, len(calls)))()
    keep = []
    for i, c in enumerate(calls):
        hm = c.get("head_map")
        hm_arr = None if hm is None else _i32(hm)
        keep.append(hm_arr)
        arr[i] = KvqDecodeDesc(ctypes.pointer(c["cache"].desc), _ptr(c.get("q16")), c["n_q_heads"], c["t_q"],
                               int(c.get("causal_tail", False)), _ptr(c.get("seq_lens")), c["max_len"],
                               ctypes.cast(hm_arr, POINTER(c_int32)) if hm_arr is not None else None,
                               float(c.get("sm_scale", 1.0)), _ptr(c.get("out")), _ptr(c.get("lse")),
                               _ptr(c.get("k16_new")), _ptr(c.get("v16_new")))
    return arr, keep


def kvq_decode_multi_workspace_size(calls) -> int:
    """Bytes of workspace kvq_decode_attn_multi needs for these calls."""
    arr, keep = _descs(calls)
    size = c_size_t(0)
    st = load().kvq_decode_multi_workspace_size(len(calls), arr, ctypes.byref(size))
    if st:
        raise KvqError(st, "kvq_decode_multi_workspace_size")
    return int(size.value)


def kvq_decode_attn_multi(calls, workspace, stream=None) -> None:
    """kvq_decode_attn_multi of include/kvq.h: several decode calls (list of
    dicts, see _descs) in one launch."""
    arr, keep = _descs(calls)
    st = load().kvq_decode_attn_multi(len(calls), arr, _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                      _stream(stream))
    if st:
        raise KvqError(st, "kvq_decode_attn_multi")


class MultiCall:
    """A prepared kvq_decode_attn_multi: the descriptor array is built once and
    each call only passes the stream (the caches' host tables are read at call
    time, so appends between calls are seen)."""

    def __init__(self, calls, workspace=None):
        self.calls = list(calls)
        self.arr, self._keep = _descs(self.calls)
        self.ws = workspace

    def workspace_size(self) -> int:
        size = c_size_t(0)
        st = load().kvq_decode_multi_workspace_size(len(self.calls), self.arr, ctypes.byref(size))
        if st:
            raise KvqError(st, "kvq_decode_multi_workspace_size")
        return int(size.value)

    def __call__(self, stream=None):
        ws = self.ws
        st = load().kvq_decode_attn_multi(len(self.calls), self.arr, _ptr(ws), 0 if ws is None else ws.numel(),
                                          _stream(stream))
        if st:
            raise KvqError(st, "kvq_decode_attn_multi")


def kvq_decode_attn_noalloc(cache: Cache, q16: torch.Tensor, n_q_heads: int, t_q: int, causal_tail: bool,
                            seq_lens: torch.Tensor, max_len: int, head_map, sm_scale: float, out: torch.Tensor,
                            lse: torch.Tensor, stream=None) -> None:
    """kvq_decode_attn_noalloc of include/kvq.h: no workspace argument; the split
    partials use the library's fixed device scratch (see the header for the
    size limit, the first-call set-up and the no-overlap rule)."""
    hm = None if head_map is None else _i32(head_map)
    st = load().kvq_decode_attn_noalloc(ctypes.byref(cache.desc), _ptr(q16), n_q_heads, t_q, int(causal_tail),
                                        _ptr(seq_lens), max_len, hm, float(sm_scale), _ptr(out), _ptr(lse),
                                        _stream(stream))
    if st:
        raise KvqError(st, "kvq_decode_attn_noalloc")


DUMP_KERNELS = ("split", "tcgen05")


def kvq_debug_qk(cache: Cache, q16, n_q_heads, t_q, seq_lens, max_len, head_map, q_codes, q_scales, scores,
                 stream=None) -> str:
    """kvq_debug_qk test hook of include/kvq.h; returns the kernel that
    produced the dumps ("split" or "tcgen05")."""
    hm = None if head_map is None else _i32(head_map)
    kern = c_int32(-1)
    st = load().kvq_debug_qk(ctypes.byref(cache.desc), _ptr(q16), n_q_heads, t_q, _ptr(seq_lens), max_len, hm,
                             _ptr(q_codes), _ptr(q_scales), _ptr(scores), ctypes.byref(kern), _stream(stream))
    if st:
        raise KvqError(st, "kvq_debug_qk")
    return DUMP_KERNELS[kern.value]


def kvq_wait_timeouts() -> int:
    """kvq_wait_timeouts of include/kvq.h: the device's count of attention-kernel
    copy waits that gave up (0 in every correct run)."""
    n = ctypes.c_uint32(0)
    st = load().kvq_wait_timeouts(ctypes.byref(n))
    if st not in (0, KVQ_ERR_TIMEOUT):
        raise KvqError(st, "kvq_wait_timeouts")
    return int(n.value)


def layout_model_default() -> KvqLayoutModel:
    """kvq_layout_model_default of include/kvq.h."""
    m = KvqLayoutModel()
    st = load().kvq_layout_model_default(ctypes.byref(m))
    if st:
        raise KvqError(st, "kvq_layout_model_default")
    return m


def layout_cost(layout: int, v_type: int, n_tokens: int, model: KvqLayoutModel | None = None) -> float:
    """kvq_layout_cost of include/kvq.h (microseconds per kv head)."""
    c = ctypes.c_double(0.0)
    st = load().kvq_layout_cost(layout, v_type, n_tokens, None if model is None else ctypes.byref(model),
                                ctypes.byref(c))
    if st:
        raise KvqError(st, "kvq_layout_cost")
    return c.value


def choose_layout(k_type: int, v_type: int, n_tokens: int, model: KvqLayoutModel | None = None) -> int:
    """kvq_choose_layout of include/kvq.h."""
    out = c_int32(-1)
    st = load().kvq_choose_layout(k_type, v_type, n_tokens, None if model is None else ctypes.byref(model),
                                  ctypes.byref(out))
    if st:
        raise KvqError(st, "kvq_choose_layout")
    return out.value


def kvq_reset_wait_timeouts() -> None:
    """kvq_reset_wait_timeouts of include/kvq.h."""
    st = load().kvq_reset_wait_timeouts()
    if st:
        raise KvqError(st, "kvq_reset_wait_timeouts")


def kvq_debug_lose_stage(cache: Cache, q16: torch.Tensor, n_q_heads: int, t_q: int, causal_tail: bool,
                         seq_lens: torch.Tensor, max_len: int, head_map, sm_scale: float, out: torch.Tensor,
                         lse: torch.Tensor, workspace: torch.Tensor | None, stream=None) -> None:
    """kvq_debug_lose_stage test hook of include/kvq.h (arguments as
    kvq_decode_attn)."""
    hm = None if head_map is None else _i32(head_map)
    st = load().kvq_debug_lose_stage(ctypes.byref(cache.desc), _ptr(q16), n_q_heads, t_q, int(causal_tail),
                                     _ptr(seq_lens), max_len, hm, float(sm_scale), _ptr(out), _ptr(lse),
                                     _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                     _stream(stream))
    if st:
        raise KvqError(st, "kvq_debug_lose_stage")


PLAN_KERNELS = ("split", "prefill")


def kvq_debug_plan(calls, n_sms: int, ctas_per_sm=(1, 2, 2, 2), max_out: int = 64):
    """kvq_debug_plan of include/kvq.h (test hook): the launches the decode
    call would make for `calls` (dicts as for kvq_decode_attn_multi; only the
    caches' host descriptors are read) on a described device.  Returns
    (launches as dicts, workspace bytes); the calls whose step tokens get an
    append launch of their own first are in kvq_debug_plan.n_pre_appends."""
    arr, keep = _descs(calls)
    ctas = _i32(ctas_per_sm)
    out = (KvqPlanLaunch * max(1, max_out))()
    n_out, ws, n_pre = c_int32(0), c_size_t(0), c_int32(0)
    st = load().kvq_debug_plan(len(calls), arr, int(n_sms), ctas, out, max_out, ctypes.byref(n_out),
                               ctypes.byref(ws), ctypes.byref(n_pre))
    kvq_debug_plan.n_pre_appends = int(n_pre.value)
    if st:
        raise KvqError(st, "kvq_debug_plan")
    launches = [dict(kernel=PLAN_KERNELS[r.kernel], n_tiles8=r.n_tiles8, warps=r.warps, chunk=r.chunk,
                     chunk0=r.chunk0, n_ctas=r.n_ctas, n_rows=r.n_rows) for r in out[:min(n_out.value, max_out)]]
    return launches, int(ws.value)


# ------------------------------------------------------- the paged cache --
# (include/kvq_paged.h).  Each operator comes as a prepared call (a class whose
# arguments are checked and marshalled once; calling it only passes the stream,
# and device contents are read when the kernels run) and as a function that
# makes one and calls it.

def _check(t, name, dtype, device, shape=None, contiguous=True):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise ValueError("%s must be a %s tensor" % (name, dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the call's tensors are on %s" % (name, t.device, device))
    if shape is not None and (t.dim() != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape))):
        raise ValueError("%s has shape %s, not %s" % (name, tuple(t.shape), tuple(shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows_stride(t, name, heads, device):
    """Token stride of an fp16 [tokens][heads][128] tensor whose rows are whole."""
    _check(t, name, torch.float16, device, (None, heads, HEAD_DIM), contiguous=False)
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != HEAD_DIM):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    return t.stride(0) if t.shape[0] > 1 else heads * HEAD_DIM


def _fits(**numbers):
    """The library takes these as int32; ctypes would cut them off."""
    for name, x in numbers.items():
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError("%s = %d does not fit 32 bits" % (name, x))


# The current stream's handle: torch's private call without the Stream object (3 us),
# or, in a torch that has no such call, the public one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _PreparedCall:
    """A library call with its arguments marshalled; stream: None = torch's
    current stream of the tensors' device, which must be the current device."""
    name = ""
    _own = None    # a workspace that the call allocated

    def _bind(self, device, *args):
        self.device = device
        self._index = device.index if device.type == "cuda" else None
        self._fn = fn = getattr(load(), self.name)
        # converted once: a call of a few microseconds' work is bound by its marshalling
        self._args = tuple(t(a) if isinstance(a, int) else a for t, a in zip(fn.argtypes, args))

    def _handle(self, stream):
        if self._index is None:
            raise ValueError("%s: the tensors are on %s, not on a CUDA device" % (self.name, self.device))
        if self._index != torch.cuda.current_device():
            raise ValueError("%s: the tensors are on %s, the current device is cuda:%d"
                             % (self.name, self.device, torch.cuda.current_device()))
        if stream is None:
            return _raw_stream(self._index)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _lend(self, handle):
        """The own workspace, allocated on one stream, to another: torch may have given that memory away before, to work
        still queued on the allocating stream, and may give it away again once this call is dropped."""
        stream = _stream_object(handle, self.device)
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
        self._own.record_stream(stream)
        if not capturing:
            stream.wait_event(self._own_ready)
            self._own_streams.add(handle)

    def __call__(self, stream=None):
        handle = self._handle(stream)
        if self._own is not None and handle not in self._own_streams:
            self._lend(handle)
        st = self._fn(*self._args, handle)
        if st:
            raise KvqError(st, self.name)


def _stream_object(handle, device):
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


class PagePool:
    """A pool of pages (include/kvq_paged.h): `data`, a uint8 device tensor of
    n_pages pages, given or allocated."""

    def __init__(self, n_pages: int, page_tokens: int, n_kv_heads: int, v_type: int, k_type: int = K_I8,
                 head_dim: int = HEAD_DIM, device=None, data: torch.Tensor | None = None):
        _fits(n_pages=n_pages, page_tokens=page_tokens, n_kv_heads=n_kv_heads, head_dim=head_dim, k_type=k_type, v_type=v_type)
        self.desc = KvqPages(n_pages, page_tokens, n_kv_heads, head_dim, k_type, v_type, None)
        self.n_pages, self.page_tokens, self.n_kv_heads = n_pages, page_tokens, n_kv_heads
        self.k_type, self.v_type = k_type, v_type
        self.page_bytes = page_bytes(self.desc)
        n = n_pages * self.page_bytes
        if data is None:
            device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
            data = torch.empty(n, dtype=torch.uint8, device=device)
        _check(data, "data", torch.uint8, data.device)
        if data.numel() != n:
            raise ValueError("data has %d bytes, the pool %d" % (data.numel(), n))
        self.data, self.device = data, data.device
        self.desc.data = data.data_ptr()


def page_bytes(desc: KvqPages) -> int:
    """kvq_page_bytes of include/kvq_paged.h."""
    n = c_size_t(0)
    st = load().kvq_page_bytes(ctypes.byref(desc), ctypes.byref(n))
    if st:
        raise KvqError(st, "kvq_page_bytes")
    return int(n.value)


def _table(t, n_seqs, device):
    """(stride, columns) of an int32 block table whose rows are whole."""
    _check(t, "block_table", torch.int32, device, (n_seqs, None), contiguous=False)
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("block_table: the entries of a row must be contiguous")
    stride = t.stride(0) if n_seqs > 1 else t.shape[1]
    _fits(n_seqs=n_seqs, max_blocks=t.shape[1], table_stride=stride)
    return stride, t.shape[1]


class PageTablesCall(_PreparedCall):
    """kvq_page_tables of include/kvq_paged.h, prepared.  lens, n_new, lens_out,
    status: int32 [n_seqs]; free_pages int32 [n_pages]; n_free, n_free_out int32
    [1]; block_table int32 [n_seqs][max_blocks] (rows may be strided); q_start
    int32 [n_seqs + 1]; slots int32 [n_tokens].  lens_out may be lens and
    n_free_out may be n_free."""
    name = "kvq_page_tables"

    def __init__(self, page_tokens: int, n_pages: int, lens, n_new, free_pages, n_free, block_table, lens_out,
                 n_free_out, q_start, slots, status):
        n, dev = lens.shape[0], lens.device
        for t, what, size in ((lens, "lens", n), (n_new, "n_new", n), (free_pages, "free_pages", n_pages),
                              (n_free, "n_free", 1), (lens_out, "lens_out", n), (n_free_out, "n_free_out", 1),
                              (q_start, "q_start", n + 1), (slots, "slots", None), (status, "status", n)):
            _check(t, what, torch.int32, dev, (size,))
        stride, cols = _table(block_table, n, dev)
        _fits(page_tokens=page_tokens, n_pages=n_pages, n_tokens=slots.shape[0])
        self._keep = (lens, n_new, free_pages, n_free, block_table, lens_out, n_free_out, q_start, slots, status)
        self._bind(dev, n, page_tokens, n_pages, _ptr(lens), _ptr(n_new), _ptr(free_pages), _ptr(n_free),
                   _ptr(block_table), stride, cols, _ptr(lens_out), _ptr(n_free_out), _ptr(q_start), _ptr(slots),
                   slots.shape[0], _ptr(status))


def kvq_page_tables(page_tokens: int, n_pages: int, lens, n_new, free_pages, n_free, block_table, lens_out, n_free_out,
                    q_start, slots, status, stream=None) -> None:
    """kvq_page_tables of include/kvq_paged.h (arguments as PageTablesCall)."""
    PageTablesCall(page_tokens, n_pages, lens, n_new, free_pages, n_free, block_table, lens_out, n_free_out, q_start,
                   slots, status)(stream)


class PagedAppendCall(_PreparedCall):
    """kvq_paged_append of include/kvq_paged.h, prepared.  k16, v16: fp16
    [tokens][kv heads][128] with the same token stride (views into a fused
    projection's output will do); slots int32 [tokens]."""
    name = "kvq_paged_append"

    def __init__(self, pool: PagePool, k16, v16, slots):
        n = slots.shape[0]
        _check(slots, "slots", torch.int32, pool.device, (n,))
        stride = _rows_stride(k16, "k16", pool.n_kv_heads, pool.device)
        if _rows_stride(v16, "v16", pool.n_kv_heads, pool.device) != stride or k16.shape[0] != n or v16.shape[0] != n:
            raise ValueError("k16, v16 and slots must have one row per token and k16, v16 the same token stride")
        _fits(n_tokens=n)
        self._keep = (pool, k16, v16, slots)
        self._bind(pool.device, ctypes.byref(pool.desc), _ptr(k16), _ptr(v16), stride, _ptr(slots), n)


def kvq_paged_append(pool: PagePool, k16, v16, slots, stream=None) -> None:
    """kvq_paged_append of include/kvq_paged.h (arguments as PagedAppendCall)."""
    PagedAppendCall(pool, k16, v16, slots)(stream)


def _out_type(t, name):
    if t.dtype not in (torch.float32, torch.float16):
        raise ValueError("%s must be float32 or float16" % name)
    return OUT_F16 if t.dtype == torch.float16 else OUT_F32


class PagedGatherCall(_PreparedCall):
    """kvq_paged_gather of include/kvq_paged.h, prepared.  slots int32 [tokens];
    k_out, v_out fp32 or fp16 [tokens][kv heads][128]."""
    name = "kvq_paged_gather"

    def __init__(self, pool: PagePool, slots, k_out, v_out):
        n = slots.shape[0]
        _check(slots, "slots", torch.int32, pool.device, (n,))
        ot = _out_type(k_out, "k_out")
        for t, what in ((k_out, "k_out"), (v_out, "v_out")):
            _check(t, what, k_out.dtype, pool.device, (n, pool.n_kv_heads, HEAD_DIM))
        _fits(n_tokens=n)
        self._keep = (pool, slots, k_out, v_out)
        self._bind(pool.device, ctypes.byref(pool.desc), _ptr(slots), n, ot, _ptr(k_out), _ptr(v_out))


def kvq_paged_gather(pool: PagePool, slots, k_out, v_out, stream=None) -> None:
    """kvq_paged_gather of include/kvq_paged.h (arguments as PagedGatherCall)."""
    PagedGatherCall(pool, slots, k_out, v_out)(stream)


class PagedAttnCall(_PreparedCall):
    """kvq_paged_attn of include/kvq_paged.h, prepared.  q16: fp16
    [tokens][q heads][128] (tokens may be strided); q_start int32 [n_seqs + 1];
    max_q: the most rows one sequence has; seq_lens int32 [n_seqs]; block_table
    int32 [n_seqs][max_blocks] (rows may be strided); out fp32 or fp16
    [tokens][q heads][128]; lse fp32 [tokens][q heads] or None; workspace: a
    uint8 device tensor of workspace_size() bytes (None: one is allocated with
    the call and kept with it; calls that may overlap need one each).  A call's
    own workspace may be used on any stream: the first call on another stream
    than it was allocated on waits for that one's work so far.  Not in a capture,
    which cannot wait (torch.cuda.graph synchronizes before it begins); and a
    graph needs the call kept for as long as it is replayed."""
    name = "kvq_paged_attn"

    def __init__(self, pool: PagePool, q16, q_start, max_q: int, seq_lens, block_table, causal: bool, sm_scale: float,
                 out, lse=None, head_map=None, workspace=None):
        n, dev = seq_lens.shape[0], pool.device
        heads = q16.shape[1] if q16.dim() == 3 else 0
        stride = _rows_stride(q16, "q16", heads, dev)
        tokens = q16.shape[0]
        _check(seq_lens, "seq_lens", torch.int32, dev, (n,))
        _check(q_start, "q_start", torch.int32, dev, (n + 1,))
        ts, cols = _table(block_table, n, dev)
        ot = _out_type(out, "out")
        _check(out, "out", out.dtype, dev, (tokens, heads, HEAD_DIM))
        if lse is not None:
            _check(lse, "lse", torch.float32, dev, (tokens, heads))
        if head_map is not None and len(head_map) != heads:
            raise ValueError("head_map must list a kv head for each query head")
        max_q = int(max_q)
        _fits(max_q=max_q, n_tokens=tokens, n_q_heads=heads)
        if head_map is not None:
            head_map = [int(h) for h in head_map]
            _fits(**{"head_map[%d]" % i: h for i, h in enumerate(head_map)})
        hm = None if head_map is None else _i32(head_map)
        self.desc = KvqPagedDesc(ctypes.pointer(pool.desc), q16.data_ptr(), stride, heads, tokens, n, max_q,
                                 q_start.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), ts, cols,
                                 int(causal), None if hm is None else ctypes.cast(hm, POINTER(c_int32)),
                                 float(sm_scale), ot, out.data_ptr(), None if lse is None else lse.data_ptr())
        if workspace is None:
            size = self.workspace_size()
            workspace = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
            if size:
                at = torch.cuda.current_stream(dev)
                self._own, self._own_ready, self._own_streams = workspace, torch.cuda.Event(), {at.cuda_stream}
                if not torch.cuda.is_current_stream_capturing():
                    self._own_ready.record(at)
        else:
            _check(workspace, "workspace", torch.uint8, dev)
        self._keep = (pool, q16, q_start, seq_lens, block_table, out, lse, hm, workspace)
        self._bind(dev, ctypes.byref(self.desc), _ptr(workspace), 0 if workspace is None else workspace.numel())

    def workspace_size(self) -> int:
        size = c_size_t(0)
        st = load().kvq_paged_attn_workspace_size(ctypes.byref(self.desc), ctypes.byref(size))
        if st:
            raise KvqError(st, "kvq_paged_attn_workspace_size")
        return int(size.value)


def kvq_paged_attn(pool: PagePool, q16, q_start, max_q: int, seq_lens, block_table, causal: bool, sm_scale: float, out,
                   lse=None, head_map=None, workspace=None, stream=None) -> None:
    """kvq_paged_attn of include/kvq_paged.h (arguments as PagedAttnCall)."""
    args = (pool, q16, q_start, max_q, seq_lens, block_table, causal, sm_scale, out, lse, head_map, workspace)
    if stream is None or workspace is not None or pool.device.type != "cuda":
        PagedAttnCall(*args)(stream)
        return
    # a workspace made here belongs to the stream that uses it
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    with torch.cuda.stream(_stream_object(handle, pool.device)):
        PagedAttnCall(*args)(stream)


def kvq_debug_paged_lose_copy(call: PagedAttnCall, copy: int, stream=None) -> None:
    """kvq_debug_paged_lose_copy test hook of include/kvq_paged.h, with the arguments of a prepared attention call."""
    handle = call._handle(stream)
    ws = call._keep[-1]
    st = load().kvq_debug_paged_lose_copy(ctypes.byref(call.desc), copy, _ptr(ws), 0 if ws is None else ws.numel(),
                                          handle)
    if st:
        raise KvqError(st, "kvq_debug_paged_lose_copy")
