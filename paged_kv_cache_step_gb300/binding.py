"""Thin ctypes binding of the C ABI in include/growpage.h.

Argument marshalling only: every step of the hot path runs in the sm_103a
kernels of libgrowpage.so.  There is no fallback: if the library is missing
and cannot be built, ``load()`` raises.

Module-level functions carry the C names (``gp_create``, ``gp_boundary_demand``
...), take a context as first argument and raise ``GrowPageError`` on a
non-OK status.  Tensors are passed by device pointer; PyTorch only provides
device memory and streams.
"""

from __future__ import annotations

import array
import ctypes as C
import struct
import os
import sys
from dataclasses import dataclass

import numpy as np

from . import _build_lib

GP_OK, GP_ERR_INVALID, GP_ERR_NO_PAGES, GP_ERR_NO_SLOTS = 0, 1, 2, 3
GP_ERR_CUDA, GP_ERR_TIMEOUT, GP_ERR_STATE, GP_ERR_UNSUPPORTED = 4, 5, 6, 7
GP_DTYPE_BF16, GP_DTYPE_F32 = 0, 1
GP_POLICY_GROWPAGE, GP_POLICY_FIXED, GP_POLICY_RANDOM, GP_POLICY_INVERSE, GP_POLICY_SHRINK = 0, 1, 2, 3, 4
GP_ACT_GROW, GP_ACT_COMPRESS, GP_ACT_SHRINK = 0, 1, 2
GP_METRIC_TOP_P, GP_METRIC_ENTROPY = 0, 1
GP_SCAN_AUTO, GP_SCAN_CUDA_CORE, GP_SCAN_TENSOR_CORE = 0, 1, 2
GP_SELECT_AUTO, GP_SELECT_SPECULATIVE, GP_SELECT_IN_COMPACTION = 0, 1, 2
GP_KERNEL_EMA, GP_KERNEL_PREP, GP_KERNEL_DEMAND, GP_KERNEL_COMPRESS, GP_KERNEL_ATTENTION = 0, 1, 2, 3, 4
GP_KERNEL_SELECT, GP_KERNEL_ENTROPY = 5, 6
GP_KERNEL_APPEND, GP_KERNEL_CHUNK, GP_KERNEL_WEIGHTS, GP_KERNEL_EVICT_SELECT, GP_KERNEL_EVICT = 7, 8, 9, 10, 11
GP_KERNEL_TABLES, GP_KERNEL_MAPPED, GP_KERNEL_BOUNDS, GP_KERNEL_BLOCK_SELECT, GP_KERNEL_SPARSE = 12, 13, 14, 15, 16
GP_STEP_GIVEN, GP_STEP_NO_PAGES, GP_STEP_NO_ROWS, GP_STEP_INVALID = 0, 1, 2, 3
GP_ROPE_HALF, GP_ROPE_INTERLEAVED = 0, 1
GP_ROPE_NONE, GP_ROPE_LINEAR, GP_ROPE_BANDS, GP_ROPE_RAMP = 0, 1, 2, 3
KERNEL_NAMES = {0: "ema_update", 1: "prep_queries", 2: "boundary_demand", 3: "compress_hold",
                4: "decode_attention", 5: "select", 6: "entropy", 7: "append_tokens", 8: "chunk_attention",
                9: "weights", 10: "evict_select", 11: "evict_move", 12: "build_tables", 13: "append_mapped",
                14: "block_bounds", 15: "select_blocks", 16: "sparse_attention"}

EXPORTS = [
    "gp_config_default", "gp_create", "gp_destroy", "gp_last_error", "gp_status_string",
    "gp_page_alloc", "gp_page_ref", "gp_page_unref", "gp_page_refcount", "gp_free_page_count",
    "gp_slot_acquire", "gp_slot_release", "gp_update_summaries", "gp_boundary_demand",
    "gp_boundary_demand_noalloc",
    "gp_decide", "gp_grow_page", "gp_compress_hold", "gp_shrink", "gp_compress_fill", "gp_compact_kv",
    "gp_debug_demand_k", "gp_debug_entropy",
    "gp_debug_scores", "gp_debug_probs", "gp_debug_keep_mask", "gp_read_summaries",
    "gp_set_scan_kernel", "gp_set_timing", "gp_kernel_time", "gp_reset_timing", "gp_stats",
    "gp_debug_attention_plan",
    "gp_set_compaction_stream", "gp_wait_compaction", "gp_decode_attention",
    "gp_synchronize", "gp_debug_set_wait_limit", "gp_debug_fail_next_launch", "gp_set_selection_mode",
    "gp_append_tokens", "gp_decode_attention_weighted", "gp_chunk_attention", "gp_evict_weighted",
    "gp_build_tables", "gp_rope_default", "gp_append_mapped", "gp_block_bounds", "gp_select_blocks", "gp_sparse_attention",
]


class GpConfig(C.Structure):
    _fields_ = [
        ("num_layers", C.c_int32), ("num_q_heads", C.c_int32), ("num_kv_heads", C.c_int32),
        ("head_dim", C.c_int32), ("page_size", C.c_int32), ("kv_dtype", C.c_int32),
        ("q_dtype", C.c_int32), ("max_slots", C.c_int32), ("num_pages", C.c_int32),
        ("max_pages_per_req", C.c_int32), ("recent_window", C.c_int32), ("k_loc", C.c_int32),
        ("reserve_pages", C.c_int32), ("policy", C.c_int32),
        ("beta_s", C.c_double), ("beta_l", C.c_double), ("p", C.c_double), ("tau", C.c_double),
        ("rope_theta", C.c_double),
        ("random_compress", C.c_double), ("shrink_threshold", C.c_double),
        ("shrink_floor_pages", C.c_int32), ("random_seed", C.c_uint32),
        ("demand_metric", C.c_int32),
    ]


class GpRequest(C.Structure):
    _fields_ = [("slot", C.c_int32), ("num_pages", C.c_int32),
                ("block_table", C.POINTER(C.c_int32)), ("pos", C.c_int64)]


class GpDemand(C.Structure):
    _fields_ = [("sum_k_short", C.c_int64), ("sum_k_long", C.c_int64),
                ("num_candidates", C.c_int32), ("num_units", C.c_int32), ("delta", C.c_double),
                ("eff_short", C.c_double), ("eff_long", C.c_double)]


class GpAction(C.Structure):
    _fields_ = [("kind", C.c_int32), ("fallback", C.c_int32), ("forced", C.c_int32)]


class GpStats(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("demand_calls", "demand_requests", "grow", "compress",
                                          "fallback", "forced_grow", "cow_pages", "moved_rows",
                                          "shrink")]


class GpRope(C.Structure):
    _fields_ = [("layout", C.c_int32), ("rotary_dim", C.c_int32), ("scaling", C.c_int32), ("original_length", C.c_int32),
                ("theta", C.c_double), ("factor", C.c_double), ("low_turns", C.c_double), ("high_turns", C.c_double),
                ("amplitude", C.c_double)]


class GrowPageError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


_LIB = None


def library_path() -> str:
    return _build_lib.LIB


def load(build_if_missing: bool = True):
    """Load libgrowpage.so (building it in-tree with nvcc if absent)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build_lib.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"native library {path} is missing; run __graft_entry__.build()")
        _build_lib.build()
    lib = C.CDLL(path)
    P, I32, I64 = C.c_void_p, C.c_int32, C.c_int64
    PI32 = C.POINTER(C.c_int32)
    sig = {
        "gp_config_default": (I32, [C.POINTER(GpConfig)]),
        "gp_create": (I32, [C.POINTER(GpConfig), P, P, P, C.POINTER(P)]),
        "gp_destroy": (I32, [P]),
        "gp_last_error": (C.c_char_p, [P]),
        "gp_status_string": (C.c_char_p, [I32]),
        "gp_page_alloc": (I32, [P, PI32]),
        "gp_page_ref": (I32, [P, I32]),
        "gp_page_unref": (I32, [P, I32]),
        "gp_page_refcount": (I32, [P, I32, PI32]),
        "gp_free_page_count": (I32, [P, PI32]),
        "gp_slot_acquire": (I32, [P, PI32]),
        "gp_slot_release": (I32, [P, I32]),
        "gp_update_summaries": (I32, [P, I32, P, P, P]),
        "gp_boundary_demand": (I32, [P, I32, C.POINTER(GpRequest), P, C.POINTER(GpDemand)]),
        "gp_boundary_demand_noalloc": (I32, [P, I32, C.POINTER(GpRequest), P, C.POINTER(GpDemand), P]),
        "gp_decide": (I32, [P, I32, C.POINTER(GpRequest), C.POINTER(GpDemand), C.POINTER(GpAction)]),
        "gp_grow_page": (I32, [P, C.POINTER(GpRequest)]),
        "gp_compress_hold": (I32, [P, I32, C.POINTER(GpRequest)]),
        "gp_shrink": (I32, [P, I32, C.POINTER(GpRequest)]),
        "gp_compress_fill": (I32, [P, I32, C.POINTER(GpRequest)]),
        "gp_compact_kv": (I32, [P, I32, C.POINTER(GpRequest), P]),
        "gp_debug_demand_k": (I32, [P, I32, P]),
        "gp_debug_entropy": (I32, [P, I32, P]),
        "gp_debug_scores": (I32, [P, I32, P]),
        "gp_debug_probs": (I32, [P, I32, P]),
        "gp_debug_keep_mask": (I32, [P, I32, P]),
        "gp_read_summaries": (I32, [P, I32, P]),
        "gp_set_scan_kernel": (I32, [P, I32]),
        "gp_debug_attention_plan": (I32, [P, I32, P, I32, I32, P, P, P]),
        "gp_set_timing": (I32, [P, I32]),
        "gp_kernel_time": (I32, [P, I32, C.POINTER(C.c_double), C.POINTER(I64)]),
        "gp_reset_timing": (I32, [P]),
        "gp_stats": (I32, [P, C.POINTER(GpStats)]),
        "gp_set_compaction_stream": (I32, [P, P]),
        "gp_wait_compaction": (I32, [P, P]),
        "gp_decode_attention": (I32, [P, I32, I32, C.POINTER(GpRequest), P, P, P, P]),
        "gp_synchronize": (I32, [P]),
        "gp_debug_set_wait_limit": (I32, [P, I32, I64]),
        "gp_debug_fail_next_launch": (I32, [P, I32]),
        "gp_set_selection_mode": (I32, [P, I32]),
        "gp_append_tokens": (I32, [P, I32, I32, P, P, P, P, P, P, P, P]),
        "gp_decode_attention_weighted": (I32, [P, I32, I32, P, P, P, P, P, P]),
        "gp_chunk_attention": (I32, [P, I32, I32, P, P, P, P, P, P]),
        "gp_evict_weighted": (I32, [P, I32, C.POINTER(GpRequest), P, P, P]),
    }
    step = {
        "gp_build_tables": (I32, [P, P, P, P, P, I32, P, P, P]),
        "gp_rope_default": (I32, [C.POINTER(GpRope)]),
        "gp_append_mapped": (I32, [P, I32, P, C.POINTER(GpRope), P, I64, P, I64, P, I64, P]),
        "gp_block_bounds": (I32, [P, I32, P, I32, P, P]),
        "gp_select_blocks": (I32, [P, I32, P, I32, I32, I32, I32, P, P, P, P]),
        "gp_sparse_attention": (I32, [P, I32, P, I32, I32, P, P, P]),
    }
    if hasattr(lib, "gp_build_tables"):  # one linked without sparse.cpp has none of them
        sig.update(step)
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _check(ctx, st: int):
    if st != GP_OK:
        lib = load()
        msg = lib.gp_last_error(ctx).decode() if ctx else lib.gp_status_string(st).decode()
        raise GrowPageError(st, msg or lib.gp_status_string(st).decode())


def _ptr(t) -> int:
    """Device (or host) address of a tensor / numpy array, or 0."""
    if t is None:
        return 0
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return int(t)


class _Buffers:
    """What the buffers of a context's calls hold: the types of queries and of keys,
    the elements of a packed row of each and of the accumulated weights."""

    def __init__(self, cfg, device):
        self._codes = cfg.q_dtype, cfg.kv_dtype
        self.q_row, self.kv_row = cfg.num_q_heads * cfg.head_dim, cfg.num_kv_heads * cfg.head_dim
        self.weights = cfg.num_layers * cfg.max_slots * cfg.num_kv_heads * cfg.max_pages_per_req * cfg.page_size
        self.device = device
        self.d, self.layers, self.hkv, self.pages = cfg.head_dim, cfg.num_layers, cfg.num_kv_heads, cfg.num_pages
        self.slots, self.tables = cfg.max_slots, cfg.max_slots * cfg.max_pages_per_req
        self.q = self.kv = self.f32 = self.u8 = self.i8 = self.i32 = self.i64 = None  # torch's types, once a tensor is met

    def know_types(self):
        import torch  # loaded: a tensor of it is being looked at
        self.f32, self.u8 = torch.float32, torch.uint8
        self.i8, self.i32, self.i64 = torch.int8, torch.int32, torch.int64
        self.q, self.kv = (torch.float32 if x == GP_DTYPE_F32 else torch.bfloat16 for x in self._codes)


class _Unknown:
    """_Buffers of a context that gp_create here has not made: nothing is known."""
    q_row = kv_row = weights = d = layers = hkv = pages = slots = tables = 0
    device = q = kv = f32 = u8 = i8 = i32 = i64 = None


def _held(ctx):
    held = getattr(ctx, "buffers", _Unknown)
    if held.f32 is None and held is not _Unknown and "torch" in sys.modules:
        held.know_types()
    return held


def _dense(held, t, dtype, count) -> int:
    """_ptr of a buffer that kernels read or write as packed rows: a tensor is
    contiguous, on the engine's device, of the type that the call takes there and
    holds the elements of its rows, or more."""
    if t is None:
        return 0
    try:  # in as few looks at the tensor as it takes: half of a small call's time is here
        if t.dtype is dtype and t.numel() >= count and t.get_device() == held.device and t.is_contiguous():
            return t.data_ptr()
        placed = t.is_contiguous() and t.is_cuda
    except AttributeError:  # no tensor
        if not isinstance(t, np.ndarray):
            return _ptr(t)
        placed = False
    if not placed:
        raise GrowPageError(GP_ERR_INVALID, "a buffer must be a contiguous tensor on a CUDA device, or its address")
    if held is not _Unknown:
        if t.numel() < count or (t.dtype is not dtype and not (dtype is held.u8 and str(t.dtype) == "torch.bool")):
            raise GrowPageError(GP_ERR_INVALID, f"a buffer of {t.numel()} {t.dtype}, where the call takes {count} {dtype}")
        if held.device is not None and t.get_device() != held.device:
            raise GrowPageError(GP_ERR_INVALID, f"a buffer on device {t.get_device()}, the caches are on device {held.device}")
    return t.data_ptr()


def _weights(held, t) -> int:
    """_dense of the accumulated weights, which have one size."""
    at = _dense(held, t, held.f32, held.weights)
    if held.weights and at and hasattr(t, "numel") and t.numel() != held.weights:
        raise GrowPageError(GP_ERR_INVALID, f"{t.numel()} weights, where the engine has {held.weights}")
    return at


# ---------------------------------------------------------------------------
# requests
# ---------------------------------------------------------------------------

# gp_request packed field by field: {int32 slot, int32 num_pages, pointer
# block_table, int64 pos}, checked against the ctypes layout at import.
_REQ_PACK = struct.Struct("=iiQq")
assert (_REQ_PACK.size == C.sizeof(GpRequest) and GpRequest.slot.offset == 0 and GpRequest.num_pages.offset == 4
        and GpRequest.block_table.offset == 8 and GpRequest.pos.offset == 16), "gp_request layout"


class Request:
    """A request as the scheduler holds it: slot, block table (host), position.
    Its gp_request record is packed when a field changes, not on every call."""

    def __init__(self, slot: int, pages, pos: int, capacity: int):
        self._slot, self._pos = int(slot), int(pos)
        pages = list(pages)
        self._num_pages = len(pages)
        table = np.zeros(capacity, dtype=np.int32)
        table[:len(pages)] = pages
        self.table = table

    def _pack(self):
        self._raw = _REQ_PACK.pack(self._slot, self._num_pages, self._bt, self._pos)

    @property
    def slot(self):
        return self._slot

    @slot.setter
    def slot(self, v):
        self._slot = v
        self._pack()

    @property
    def num_pages(self):
        return self._num_pages

    @num_pages.setter
    def num_pages(self, v):
        self._num_pages = v
        self._pack()

    @property
    def pos(self):
        return self._pos

    @pos.setter
    def pos(self, v):
        self._pos = v
        self._pack()

    @property
    def table(self):
        return self._table

    @table.setter
    def table(self, t):
        self._table = np.ascontiguousarray(t, dtype=np.int32)
        self._bt = self._table.ctypes.data  # the C side reads and extends it in place
        self._pack()

    @property
    def pages(self):
        return self.table[:self.num_pages].tolist()


# gp_request as a numpy record, so that a call's requests are marshalled one
# field at a time instead of one ctypes attribute at a time
_REQ_DTYPE = np.dtype({"names": ["slot", "num_pages", "block_table", "pos"],
                       "formats": [np.int32, np.int32, np.uint64, np.int64],
                       "offsets": [GpRequest.slot.offset, GpRequest.num_pages.offset,
                                   GpRequest.block_table.offset, GpRequest.pos.offset],
                       "itemsize": C.sizeof(GpRequest)})

_NUM_PAGES = struct.Struct("=i")


def _marshal(reqs):
    arr = (GpRequest * max(1, len(reqs)))()
    if len(reqs):
        C.memmove(arr, _records(reqs), len(reqs) * _REQ_PACK.size)
    return arr


def _records(reqs) -> bytes:
    """The requests' records for a call that only reads them."""
    return b"".join([r._raw for r in reqs])


def _unmarshal(arr, reqs):
    if len(reqs) <= 8:
        get, size = _NUM_PAGES.unpack_from, _REQ_PACK.size
        counts = [get(arr, i * size + 4)[0] for i in range(len(reqs))]
    else:
        counts = np.frombuffer(arr, dtype=_REQ_DTYPE, count=len(reqs))["num_pages"].tolist()
    for r, p in zip(reqs, counts):
        if p != r._num_pages:
            r.num_pages = p


class _Demands(list):
    """gp_boundary_demand's results: gp_demand views into one ctypes array,
    which gp_decide passes on as it is while the list is unchanged."""

    def __init__(self, arr, n):
        super().__init__(arr[i] for i in range(n))
        self._arr = arr

    def __setitem__(self, i, v):
        self._arr = None
        super().__setitem__(i, v)

    def _whole(self, n):
        return self._arr if self._arr is not None and len(self) == n else None


# ---------------------------------------------------------------------------
# C-named wrappers
# ---------------------------------------------------------------------------

def gp_config_default(**overrides) -> GpConfig:
    cfg = GpConfig()
    _check(None, load().gp_config_default(C.byref(cfg)))
    for k, v in overrides.items():
        setattr(cfg, k, v)
    return cfg


def gp_create(cfg: GpConfig, k_cache=None, v_cache=None, stream=None):
    ctx = C.c_void_p()
    s = 0 if stream is None else (stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    st = load().gp_create(C.byref(cfg), _ptr(k_cache) or None, _ptr(v_cache) or None, s or None, C.byref(ctx))
    _check(None, st)
    ctx.buffers = _Buffers(cfg, k_cache.get_device() if hasattr(k_cache, "get_device") else None)
    return ctx


def gp_destroy(ctx):
    _check(None, load().gp_destroy(ctx))


def gp_page_alloc(ctx) -> int:
    p = C.c_int32()
    _check(ctx, load().gp_page_alloc(ctx, C.byref(p)))
    return p.value


def gp_page_ref(ctx, page: int):
    _check(ctx, load().gp_page_ref(ctx, page))


def gp_page_unref(ctx, page: int):
    _check(ctx, load().gp_page_unref(ctx, page))


def gp_page_refcount(ctx, page: int) -> int:
    rc = C.c_int32()
    _check(ctx, load().gp_page_refcount(ctx, page, C.byref(rc)))
    return rc.value


def gp_free_page_count(ctx) -> int:
    n = C.c_int32()
    _check(ctx, load().gp_free_page_count(ctx, C.byref(n)))
    return n.value


def gp_slot_acquire(ctx) -> int:
    s = C.c_int32()
    _check(ctx, load().gp_slot_acquire(ctx, C.byref(s)))
    return s.value


def gp_slot_release(ctx, slot: int):
    _check(ctx, load().gp_slot_release(ctx, slot))


def gp_update_summaries(ctx, n: int, slots_dev, q_dev, first_dev):
    _check(ctx, load().gp_update_summaries(ctx, n, _ptr(slots_dev), _ptr(q_dev), _ptr(first_dev)))


def gp_boundary_demand(ctx, reqs, q_cur_dev):
    arr = _marshal(reqs)
    out = (GpDemand * max(1, len(reqs)))()
    _check(ctx, load().gp_boundary_demand(ctx, len(reqs), arr, _ptr(q_cur_dev), out))
    return _Demands(out, len(reqs))


def gp_boundary_demand_noalloc(ctx, reqs, q_cur_dev, k_units=None):
    """No-allocation variant; k_units (host int32 [n][L*Hkv][2]) is optional."""
    arr = _marshal(reqs)
    out = (GpDemand * max(1, len(reqs)))()
    _check(ctx, load().gp_boundary_demand_noalloc(ctx, len(reqs), arr, _ptr(q_cur_dev), out,
                                                  _ptr(k_units) or None))
    return [out[i] for i in range(len(reqs))]


def gp_decide(ctx, reqs, demand):
    arr = _marshal(reqs)
    dem = demand._whole(len(reqs)) if isinstance(demand, _Demands) else None
    if dem is None:
        dem = (GpDemand * max(1, len(reqs)))(*demand)
    out = (GpAction * max(1, len(reqs)))()
    _check(ctx, load().gp_decide(ctx, len(reqs), arr, dem, out))
    return [out[i] for i in range(len(reqs))]


def gp_grow_page(ctx, req: Request):
    if req.num_pages >= len(req.table):
        raise GrowPageError(GP_ERR_INVALID, "block table is full (Python capacity)")
    arr = _marshal([req])
    st = load().gp_grow_page(ctx, arr)
    _unmarshal(arr, [req])
    _check(ctx, st)


def gp_compress_hold(ctx, reqs):
    arr = _marshal(reqs)
    st = load().gp_compress_hold(ctx, len(reqs), arr)
    _unmarshal(arr, reqs)
    _check(ctx, st)


def gp_shrink(ctx, reqs):
    arr = _marshal(reqs)
    st = load().gp_shrink(ctx, len(reqs), arr)
    _unmarshal(arr, reqs)
    _check(ctx, st)


def gp_compress_fill(ctx, reqs):
    arr = _marshal(reqs)
    st = load().gp_compress_fill(ctx, len(reqs), arr)
    _unmarshal(arr, reqs)
    _check(ctx, st)


def _stream_ptr(stream):
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def gp_set_compaction_stream(ctx, stream):
    _check(ctx, load().gp_set_compaction_stream(ctx, _stream_ptr(stream)))


def gp_wait_compaction(ctx, stream=None):
    _check(ctx, load().gp_wait_compaction(ctx, _stream_ptr(stream)))


def gp_decode_attention(ctx, layer: int, reqs, num_tokens, q_dev, first_dev, out_dev):
    """One layer of decode attention with the summary update fused in.
    num_tokens: host int32 per request; q_dev [n][Hq][d]; out_dev fp32 [n][Hq][d]."""
    arr = _marshal(reqs)
    nt = np.ascontiguousarray(np.asarray(num_tokens, dtype=np.int32))
    _check(ctx, load().gp_decode_attention(ctx, layer, len(reqs), arr, nt.ctypes.data, _ptr(q_dev),
                                           _ptr(first_dev), _ptr(out_dev)))


def _counts(reqs, *lists):
    """Host int32 arrays of per-request counts, one entry a request."""
    out = []
    for x in lists:
        try:
            if type(x) is list or type(x) is tuple:
                a = array.array("i", x)
                n = len(a)
            else:
                a = np.asarray(x)
                if a.dtype != np.int32:  # counted one by one: a cast would cut bits off
                    a = np.asarray(array.array("i", a.ravel().tolist()), dtype=np.int32).reshape(a.shape)
                a = np.ascontiguousarray(a)
                n = len(a) if a.ndim == 1 else -1
        except (OverflowError, TypeError) as err:
            raise GrowPageError(GP_ERR_INVALID, f"counts must be whole numbers of 32 bits: {err}") from None
        if n != len(reqs):
            raise GrowPageError(GP_ERR_INVALID, f"{len(reqs)} requests, {n} counts")
        out.append(a)
    return out


def _host(a) -> int:
    """Host address of a counts array."""
    return a.buffer_info()[0] if type(a) is array.array else a.ctypes.data


def _total(a) -> int:
    return sum(a) if type(a) is array.array else int(a.sum(dtype=np.int64))


def gp_append_tokens(ctx, layer: int, reqs, num_cached, num_new, q_dev, k_dev, v_dev, q_rot_dev, weights_dev=None):
    """New tokens of one layer into the cache: rotated keys, values, rotated
    queries, cleared weights.  num_cached, num_new: host int32 per request;
    q_dev, q_rot_dev [rows][Hq][d] (both None: keys and values alone);
    k_dev, v_dev [rows][Hkv][d], rows packed request after request."""
    nc, nn = _counts(reqs, num_cached, num_new)
    held, rows = _held(ctx), _total(nn)
    q, kv = rows * held.q_row, rows * held.kv_row
    _check(ctx, load().gp_append_tokens(ctx, layer, len(reqs), _records(reqs), _host(nc), _host(nn),
                                        _dense(held, q_dev, held.q, q), _dense(held, k_dev, held.kv, kv), _dense(held, v_dev, held.kv, kv),
                                        _dense(held, q_rot_dev, held.q, q), _weights(held, weights_dev)))


def gp_decode_attention_weighted(ctx, layer: int, reqs, num_tokens, q_dev, first_dev, out_dev, weights_dev):
    """gp_decode_attention that adds its softmax weights to weights_dev
    (fp32 [L][max_slots][Hkv][max_pages_per_req * 256]); first_dev may be None."""
    nt, = _counts(reqs, num_tokens)
    n = len(reqs)
    held = _held(ctx)
    q = n * held.q_row
    _check(ctx, load().gp_decode_attention_weighted(ctx, layer, n, _records(reqs), _host(nt), _dense(held, q_dev, held.q, q),
                                                    _dense(held, first_dev, held.u8, n), _dense(held, out_dev, held.f32, q),
                                                    _weights(held, weights_dev)))


def gp_chunk_attention(ctx, layer: int, reqs, num_cached, num_new, q_dev, out_dev, weights_dev=None):
    """Causal attention of each request's num_new last tokens over its cache;
    q_dev (rotated) and out_dev [rows][Hq][d] of q_dtype, packed.  Added weights
    stay: of drafted tokens, add the accepted ones' in a second call."""
    nc, nn = _counts(reqs, num_cached, num_new)
    held = _held(ctx)
    q = _total(nn) * held.q_row
    _check(ctx, load().gp_chunk_attention(ctx, layer, len(reqs), _records(reqs), _host(nc), _host(nn),
                                          _dense(held, q_dev, held.q, q), _dense(held, out_dev, held.q, q), _weights(held, weights_dev)))


def gp_evict_weighted(ctx, reqs, num_tokens, keep_tokens, weights_dev):
    """Keep each request's recent window and its tokens of most accumulated
    weight, keep_tokens in all, per (layer, KV head); K, V and weights are
    compacted in order.  Rewrites the requests' tables (copy-on-write)."""
    nt, nk = _counts(reqs, num_tokens, keep_tokens)
    arr = _marshal(reqs)
    st = load().gp_evict_weighted(ctx, len(reqs), arr, _host(nt), _host(nk), _weights(_held(ctx), weights_dev))
    _unmarshal(arr, reqs)
    _check(ctx, st)


# gp_step packed field by field: {int32 n, int32 max_rows, nine pointers}
_STEP_PACK = struct.Struct("=ii9Q")


class Step:
    """The device arrays of a step (gp_step): tensors, checked here once against the
    context, or addresses, with n and max_rows then given.  The step keeps the
    tensors alive."""

    def __init__(self, ctx, *, slots, num_cached, num_new, pos, tables, row0, row_req, slot_map, positions, n=None,
                 max_rows=None):
        self.n = int(len(slots) if n is None else n)
        self.max_rows = int(len(row_req) if max_rows is None else max_rows)
        h, n, rows = _held(ctx), self.n, self.max_rows
        self.arrays = (slots, num_cached, num_new, pos, tables, row0, row_req, slot_map, positions)
        if hasattr(tables, "numel") and h.tables and tables.numel() != h.tables:
            raise GrowPageError(GP_ERR_INVALID, f"block tables of {tables.numel()} entries, where the engine has {h.tables}")
        self._raw = _STEP_PACK.pack(
            n, rows, _dense(h, slots, h.i32, n), _dense(h, num_cached, h.i32, n), _dense(h, num_new, h.i32, n),
            _dense(h, pos, h.i64, n), _dense(h, tables, h.i32, h.tables), _dense(h, row0, h.i32, n + 1),
            _dense(h, row_req, h.i32, rows), _dense(h, slot_map, h.i64, rows), _dense(h, positions, h.i64, rows))


def _strided(held, t, dtype, rows, row):
    """Address of rows of packed heads and the elements between their starts: a
    tensor [rows, heads, d] or [rows, heads * d], dense within a row."""
    if t is None:
        return 0, 0
    try:  # heads side by side, in as few looks at the tensor as it takes
        shape, (apart, head, one) = t.shape, t.stride()
        if (one == 1 and head == shape[2] and shape[1] * head == row and shape[0] >= rows and t.dtype is dtype
                and t.get_device() == held.device):
            return t.data_ptr(), apart if rows > 1 else row
    except (AttributeError, ValueError):
        pass
    if not hasattr(t, "stride") or t.dim() < 2 or rows == 0:
        return _dense(held, t, dtype, 0), row
    shape, strides = t.shape, t.stride()
    dense = 1
    for size, stride in zip(reversed(shape[1:]), reversed(strides[1:])):
        if size != 1 and stride != dense:
            raise GrowPageError(GP_ERR_INVALID, f"rows that are not dense: strides {strides}")
        dense *= size
    if not t.is_cuda or (held.device is not None and t.get_device() != held.device):
        raise GrowPageError(GP_ERR_INVALID, f"a buffer on {t.device}, the caches are on device {held.device}")
    if held is not _Unknown and (t.dtype is not dtype or dense != row or shape[0] < rows):
        raise GrowPageError(GP_ERR_INVALID, f"{shape[0]} rows of {dense} {t.dtype}, where the call takes {rows} of {row} {dtype}")
    return t.data_ptr(), strides[0] if rows > 1 else row


def gp_rope_default(**overrides) -> GpRope:
    rope = GpRope()
    _check(None, load().gp_rope_default(C.byref(rope)))
    for k, v in overrides.items():
        if k not in dict(GpRope._fields_):
            raise TypeError(f"gp_rope has no field {k}")
        setattr(rope, k, v)
    return rope


def gp_build_tables(ctx, step: Step, held_dev, num_pages_dev, free_dev, taken_in_dev, taken_dev, state_dev, num_free=None):
    """Rows, block tables, slot map and positions of a step.  held_dev, num_pages_dev:
    int32 [max_slots]; free_dev: int32 page ids (num_free of them, all by default);
    taken_in_dev (or None), taken_dev: int32 [1]; state_dev: int32 [n]."""
    h = _held(ctx)
    if num_free is None:
        num_free = 0 if free_dev is None else free_dev.numel()
    _check(ctx, load().gp_build_tables(ctx, step._raw, _dense(h, held_dev, h.i32, h.slots), _dense(h, num_pages_dev, h.i32, h.slots),
                                       _dense(h, free_dev, h.i32, num_free), num_free, _dense(h, taken_in_dev, h.i32, 1),
                                       _dense(h, taken_dev, h.i32, 1), _dense(h, state_dev, h.i32, step.n)))


def gp_append_mapped(ctx, layer: int, step: Step, rope: GpRope, q_dev, k_dev, v_dev, q_rot_dev):
    """The step's tokens of one layer into the cache, in a rotary form.  q_dev, k_dev,
    v_dev: [max_rows, heads, d], rows any multiple of 16 bytes apart; q_rot_dev
    packed.  q_dev and q_rot_dev both None: keys and values alone."""
    h, rows = _held(ctx), step.max_rows
    q, qs = _strided(h, q_dev, h.q, rows, h.q_row)
    k, ks = _strided(h, k_dev, h.kv, rows, h.kv_row)
    v, vs = _strided(h, v_dev, h.kv, rows, h.kv_row)
    _check(ctx, load().gp_append_mapped(ctx, layer, step._raw, rope, q, qs, k, ks, v, vs,
                                        _dense(h, q_rot_dev, h.q, rows * h.q_row)))


def _bounds(h, block, bounds_dev, scales_dev):
    blocks = h.layers * h.pages * h.hkv * (256 // block if block > 0 else 0)
    return _dense(h, bounds_dev, h.i8, blocks * 2 * h.d), _dense(h, scales_dev, h.f32, blocks)


def gp_block_bounds(ctx, layer: int, step: Step, block: int, bounds_dev, scales_dev):
    """Bounds of the blocks that the step's rows fall into: bounds_dev int8
    [L][num_pages][Hkv][256 / block][2][d], scales_dev fp32, one a block and head."""
    h = _held(ctx)
    _check(ctx, load().gp_block_bounds(ctx, layer, step._raw, block, *_bounds(h, block, bounds_dev, scales_dev)))


def gp_select_blocks(ctx, layer: int, step: Step, block: int, top: int, sink: int, recent: int, q_rot_dev, bounds_dev, scales_dev,
                     blocks_dev):
    """The `top` blocks of each row and KV head: the first `sink`, the last `recent`,
    and those of largest score; blocks_dev int32 [max_rows][Hkv][top]."""
    h, rows = _held(ctx), step.max_rows
    b, s = _bounds(h, block, bounds_dev, scales_dev)
    _check(ctx, load().gp_select_blocks(ctx, layer, step._raw, block, top, sink, recent, _dense(h, q_rot_dev, h.q, rows * h.q_row),
                                        b, s, _dense(h, blocks_dev, h.i32, rows * h.hkv * top)))


def gp_sparse_attention(ctx, layer: int, step: Step, block: int, top: int, q_rot_dev, blocks_dev, out_dev):
    """Attention of each row over the blocks listed for it; q_rot_dev and out_dev
    [max_rows][Hq][d] of q_dtype, blocks_dev as gp_select_blocks gives it."""
    h, rows = _held(ctx), step.max_rows
    q = rows * h.q_row
    _check(ctx, load().gp_sparse_attention(ctx, layer, step._raw, block, top, _dense(h, q_rot_dev, h.q, q),
                                           _dense(h, blocks_dev, h.i32, rows * h.hkv * top), _dense(h, out_dev, h.q, q)))


def gp_compact_kv(ctx, reqs, keep_masks_dev):
    arr = _marshal(reqs)
    st = load().gp_compact_kv(ctx, len(reqs), arr, _ptr(keep_masks_dev))
    _unmarshal(arr, reqs)
    _check(ctx, st)


def gp_debug_demand_k(ctx, req_idx: int, units: int) -> np.ndarray:
    out = np.zeros((units, 2), dtype=np.int32)
    _check(ctx, load().gp_debug_demand_k(ctx, req_idx, out.ctypes.data))
    return out


def gp_debug_entropy(ctx, req_idx: int, units: int) -> np.ndarray:
    out = np.zeros((units, 2), dtype=np.float64)
    _check(ctx, load().gp_debug_entropy(ctx, req_idx, out.ctypes.data))
    return out


def gp_debug_scores(ctx, req_idx: int, units: int, ncmp: int) -> np.ndarray:
    out = np.zeros((units, ncmp), dtype=np.float32)
    _check(ctx, load().gp_debug_scores(ctx, req_idx, out.ctypes.data))
    return out


def gp_debug_probs(ctx, req_idx: int, units: int, ndem: int) -> np.ndarray:
    out = np.zeros((units, 2, ndem), dtype=np.float32)
    _check(ctx, load().gp_debug_probs(ctx, req_idx, out.ctypes.data))
    return out


def gp_debug_keep_mask(ctx, req_idx: int, units: int, num_pages: int, page_size: int = 256) -> np.ndarray:
    out = np.zeros((units, num_pages * page_size // 32), dtype=np.uint32)
    _check(ctx, load().gp_debug_keep_mask(ctx, req_idx, out.ctypes.data))
    return out


def gp_read_summaries(ctx, slot: int, L: int, hq: int, d: int) -> np.ndarray:
    out = np.zeros((L, 2, hq, d), dtype=np.float64)
    _check(ctx, load().gp_read_summaries(ctx, slot, out.ctypes.data))
    return out



def gp_debug_attention_plan(ctx, num_tokens, sms: int) -> np.ndarray:
    """The tensor-core attention kernel's work items for these token counts on
    `sms` SMs (host only): int32 [items][8] rows (request, KV head, piece,
    pieces, first page, tiles, first item of the pair, CTA)."""
    nt = np.ascontiguousarray(np.asarray(num_tokens, dtype=np.int32))
    n_items, n_ctas = C.c_int32(0), C.c_int32(0)
    lib = load()
    lib.gp_debug_attention_plan(ctx, len(nt), nt.ctypes.data, int(sms), 0, None, C.byref(n_items), C.byref(n_ctas))
    out = np.zeros((max(n_items.value, 1), 8), dtype=np.int32)
    _check(ctx, lib.gp_debug_attention_plan(ctx, len(nt), nt.ctypes.data, int(sms), out.shape[0], out.ctypes.data,
                                            C.byref(n_items), C.byref(n_ctas)))
    return out[:n_items.value]


def gp_set_scan_kernel(ctx, kind: int):
    _check(ctx, load().gp_set_scan_kernel(ctx, int(kind)))


def gp_set_selection_mode(ctx, mode: int):
    _check(ctx, load().gp_set_selection_mode(ctx, int(mode)))


def gp_set_timing(ctx, enabled: bool):
    _check(ctx, load().gp_set_timing(ctx, int(bool(enabled))))


def gp_kernel_time(ctx, kernel: int):
    ms, n = C.c_double(), C.c_int64()
    _check(ctx, load().gp_kernel_time(ctx, kernel, C.byref(ms), C.byref(n)))
    return ms.value, n.value


def gp_reset_timing(ctx):
    _check(ctx, load().gp_reset_timing(ctx))


def gp_synchronize(ctx):
    """Wait for all engine work; raise on device-side errors of earlier calls."""
    _check(ctx, load().gp_synchronize(ctx))


def gp_debug_set_wait_limit(ctx, kernel: int, cycles: int):
    _check(ctx, load().gp_debug_set_wait_limit(ctx, int(kernel), int(cycles)))


def gp_debug_fail_next_launch(ctx, kernel: int):
    _check(ctx, load().gp_debug_fail_next_launch(ctx, int(kernel)))


def gp_stats(ctx) -> dict:
    s = GpStats()
    _check(ctx, load().gp_stats(ctx, C.byref(s)))
    return {n: getattr(s, n) for n, _ in GpStats._fields_}


@dataclass
class Shape:
    num_layers: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int

    @property
    def units(self) -> int:
        return self.num_layers * self.num_kv_heads


def unpack_mask(words: np.ndarray, n: int) -> np.ndarray:
    """uint32 keep-mask words -> bool[..., n] (bit i%32 of word i/32)."""
    w = np.asarray(words, dtype=np.uint32)
    bits = ((w[..., :, None] >> np.arange(32, dtype=np.uint32)) & 1).astype(bool)
    return bits.reshape(*w.shape[:-1], -1)[..., :n]


def pack_mask(keep: np.ndarray) -> np.ndarray:
    """bool[..., n] (n a multiple of 32) -> uint32 words."""
    k = np.asarray(keep, dtype=bool)
    k = k.reshape(*k.shape[:-1], -1, 32).astype(np.uint32)
    return (k << np.arange(32, dtype=np.uint32)).sum(axis=-1).astype(np.uint32)
