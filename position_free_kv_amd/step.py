"""ctypes binding of the serving step (include/kamera_step.h): same names, argument marshalling only.

Every computation runs in the library's HIP kernels. A `Step` is marshalled once and may be
kept between steps: its `num_tokens`, `num_queries`, `slot0`, `position0` and block tables are
read by each upload, so a decode loop changes them in place.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np

from . import abi
from .abi import Layout, Pool, _check, _ptr, _ws

APPEND, ATTEND, FIT = 1, 2, 4
REQUEST_ALL = 1
ATTEND_MAX_DIM = 1024

EXPORTED = ["kamera_step_workspace_bytes", "kamera_step_upload", "kamera_step_append", "kamera_step_attend",
            "kamera_copy_pages_workspace_bytes", "kamera_copy_pages", "kamera_compact_pages"]


class Prefix(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("slot0", ctypes.c_int32), ("num_tokens", ctypes.c_int32)]


class Request(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("slot0", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("num_queries", ctypes.c_int32), ("prefix", ctypes.c_int32), ("position0", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32)]


class StepDesc(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_void_p), ("prefixes", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("num_requests", ctypes.c_int32), ("num_prefixes", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32 * 2)]


class Plan(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("num_tokens", ctypes.c_int32), ("num_layers", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32), ("detail", ctypes.c_uint64 * 40)]
    _like = None  # what the launches' tensors have to be (set by upload)


class AppendRows(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


_REQUEST = np.dtype({"names": [n for n, _ in Request._fields_],
                     "formats": [np.uint64, np.int32, np.int32, np.int32, np.int32, np.int64, np.uint32, np.int32],
                     "offsets": [getattr(Request, n).offset for n, _ in Request._fields_],
                     "itemsize": ctypes.sizeof(Request)})
_PREFIX = np.dtype({"names": [n for n, _ in Prefix._fields_], "formats": [np.uint64, np.int32, np.int32],
                    "offsets": [getattr(Prefix, n).offset for n, _ in Prefix._fields_],
                    "itemsize": ctypes.sizeof(Prefix)})

_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        L = abi.lib()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lay, pool, plan = ctypes.POINTER(Layout), ctypes.POINTER(Pool), ctypes.POINTER(Plan)
        L.kamera_step_workspace_bytes.argtypes = [lay, ctypes.POINTER(StepDesc)]
        L.kamera_step_upload.argtypes = [lay, ctypes.POINTER(StepDesc), pool, vp, sz, vp, plan]
        L.kamera_step_append.argtypes = [plan, i32, ctypes.POINTER(AppendRows), vp]
        L.kamera_step_attend.argtypes = [plan, i32, vp, i64, vp, i64, vp, ctypes.c_float, vp]
        L.kamera_copy_pages_workspace_bytes.argtypes = [i32]
        L.kamera_copy_pages.argtypes = [lay, pool, vp, vp, i32, vp, sz, vp]
        L.kamera_compact_pages.argtypes = [lay, pool, ctypes.POINTER(vp), vp, i32, ctypes.POINTER(i32), vp, sz, vp]
        for name in EXPORTED:
            getattr(L, name).restype = sz if name.endswith("_bytes") else ctypes.c_int
        _bound = L
    return _bound


_current = None  # () -> handle of torch's current stream where there is a GPU, else False


def _stream(stream) -> Optional[int]:
    """Handle of a stream: torch's current one by default (None, the null stream, without a GPU)."""
    global _current
    if stream is None:
        if _current is None:
            _current = False
            try:
                import torch
                if torch.cuda.is_available():
                    torch.cuda.init()
                    raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice  # (current_stream() makes an object a call)
                    _current = lambda: raw(device())
            except ImportError:
                pass
        return _current() if _current else None
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def _table(t) -> np.ndarray:
    """A host int32 table, shared with the caller: what it holds at an upload is what the upload reads."""
    a = None if isinstance(t, (list, tuple)) else np.asarray(t)
    if a is None or a.dtype != np.int32 or a.ndim != 1 or not a.flags.c_contiguous:
        raise ValueError("block tables are int32 arrays of one dimension, contiguous (the library reads them in place)")
    return a


def _tables(block_tables, n: int):
    """Host int32 tables, one a request: a 2-D array (a row each) or a sequence of arrays (None: no table).
    Returns (addresses, entries, objects to keep alive)."""
    if isinstance(block_tables, np.ndarray) and block_tables.ndim == 2:
        rows, width = block_tables.shape
        if rows != n:
            raise ValueError(f"{rows} block tables for {n} requests")
        if block_tables.dtype != np.int32 or (width > 1 and block_tables.strides[1] != 4):
            raise ValueError("rows of block tables are contiguous and int32 (the library reads them in place)")
        addresses = block_tables.ctypes.data + np.arange(n, dtype=np.int64) * block_tables.strides[0]
        return addresses.astype(np.uint64), np.full(n, width, dtype=np.int64), block_tables
    keep = [None if t is None else _table(t) for t in block_tables]
    if len(keep) != n:
        raise ValueError(f"{len(keep)} block tables for {n} requests")
    return (np.array([0 if t is None else t.ctypes.data for t in keep], dtype=np.uint64),
            np.array([0 if t is None else t.size for t in keep], dtype=np.int64), keep)


class _Entries:
    """How many tokens each record's table holds entries for. The library takes a table by its address alone and reads
    what the tokens need, so a shorter one is refused here. Records that the library refuses before it reads any table
    (no address, slot0 outside a page, tokens beyond 2^31 - 4096) are left to it."""

    def __init__(self, what: str, records: np.ndarray, entries: np.ndarray):
        self._what, self._records, self._entries = what, records, entries
        self._slot0, self._tokens = records["slot0"], records["num_tokens"]
        self._page_size, self._limit = 0, entries

    def check(self, page_size: int) -> None:
        if page_size != self._page_size:
            self._page_size, self._limit = page_size, self._entries * max(page_size, 1)
        # (a sum that wraps belongs to a record that the library refuses)
        if not np.count_nonzero(self._slot0 + self._tokens > self._limit) or page_size < 1:
            return
        slot0, tokens = self._slot0.astype(np.int64), self._tokens.astype(np.int64)
        short = (tokens > 0) & (slot0 + tokens > self._limit) & (slot0 + tokens < (1 << 31) - 4096)
        short &= (self._records["block_table"] != 0) & (slot0 >= 0) & (slot0 < page_size)
        for i in np.flatnonzero(short)[:1]:
            raise ValueError(f"{self._what} {i}: {self._entries[i]} block table entries of {page_size} tokens "
                             f"for {tokens[i]} tokens from slot {slot0[i]} on")


class Step:
    """A kamera_step and the host arrays it points into.

    block_tables: a 2-D int32 array or a sequence of 1-D ones (None: a request without tokens of
    its own), a row a request, read in place by every upload (rows may be part of a wider array; other
    types are refused, as a copy would not follow the caller's changes) and as long as slot0 + num_tokens needs. The other
    request fields are scalars or one value a request. prefixes: dicts with block_table,
    num_tokens and (optionally) slot0. `requests` is the structured array the library reads.
    """

    def __init__(self, *, num_q_heads: int, block_tables, num_tokens, num_queries, slot0=0, prefix=-1,
                 prefixes: Sequence[dict] = (), position0=0, request_flags=0, positions=None, flags: int = APPEND | ATTEND):
        n = len(block_tables)
        addresses, entries, self._keep = _tables(block_tables, n)
        self.requests = np.zeros(n, _REQUEST)
        self.requests["block_table"] = addresses
        for name, value in (("slot0", slot0), ("num_tokens", num_tokens), ("num_queries", num_queries),
                            ("prefix", prefix), ("position0", position0), ("flags", request_flags)):
            self.requests[name] = value
            if (self.requests[name] != value).any():
                raise ValueError(f"{name}: a value does not fit its field")
        self._prefix_tables = [_table(p["block_table"]) for p in prefixes]
        self.prefixes = np.zeros(len(prefixes), _PREFIX)
        for i, p in enumerate(prefixes):
            self.prefixes[i] = (self._prefix_tables[i].ctypes.data, p.get("slot0", 0), p["num_tokens"])
        self._entries = [_Entries("request", self.requests, entries)] if n else []
        if len(prefixes):
            self._entries.append(_Entries("prefix", self.prefixes, np.array([t.size for t in self._prefix_tables], dtype=np.int64)))
        self._positions = positions
        self.c = StepDesc(self.requests.ctypes.data if n else None, self.prefixes.ctypes.data if len(prefixes) else None,
                          _ptr(positions), n, len(prefixes), int(num_q_heads), int(flags))


def workspace_bytes(layout: Layout, step: Step) -> int:
    """Bytes that a step needs. They do not only grow with its lengths: a buffer for the largest step serves the
    smaller ones too if FIT is among their flags."""
    return int(_lib().kamera_step_workspace_bytes(ctypes.byref(layout), ctypes.byref(step.c)))


class _Like:
    """What the tensors of a step's launches have to be: the layout's element type and widths. The library takes
    addresses and strides between tokens alone, so anything else would be read as something that it is not."""

    def __init__(self, torch, layout: Layout, num_q_heads: int):
        self.gqa = gqa = layout.family == abi.GQA
        self.dtype = torch.bfloat16 if layout.dtype == abi.BF16 else torch.float32
        self.k = layout.num_kv_heads * layout.head_dim if gqa else layout.latent_dim + layout.rope_dim
        self.dk = layout.head_dim if gqa else self.k
        self.normed = layout.head_dim if gqa else layout.latent_dim  # columns of the keys' norm
        self.heads = num_q_heads
        self.q, self.out = num_q_heads * self.dk, num_q_heads * (self.dk if gqa else layout.latent_dim)
        self.stats, self.positions = torch.float32, torch.int32


def _on_gpu(what: str, x) -> None:
    if not x.is_cuda and not x.is_pinned():
        raise ValueError(f"{what}: a tensor of {x.device}, which the GPU does not read")


def _flat(what: str, x, dtype, size: int, exactly: bool = False) -> Optional[int]:
    """Address of a packed tensor of `size` elements (or more)."""
    if x is None or isinstance(x, int):
        return x
    have = x.numel()
    if x.dtype is not dtype or not x.is_contiguous() or have < size or (exactly and have != size):
        raise ValueError(f"{what}: {tuple(x.shape)} of {x.dtype}, strides {x.stride()}; {size} packed elements of {dtype} are needed")
    _on_gpu(what, x)
    return x.data_ptr()


def upload(layout: Layout, step: Step, pool: Pool, workspace, stream=None) -> Plan:
    """Validate a step and put its description into the workspace; the plan serves every layer.
    It points into the workspace and keeps that tensor alive."""
    for tables in step._entries:
        tables.check(layout.page_size)
    like = None
    try:
        import torch
        like = _Like(torch, layout, step.c.num_q_heads)
    except ImportError:  # addresses alone
        pass
    if like is not None and step._positions is not None and step.c.flags & APPEND:
        _flat("positions", step._positions, like.positions, 3 * int(step.requests["num_queries"].sum(dtype=np.int64)))
    wp, wb = _ws(workspace)
    plan = Plan()
    _check(_lib().kamera_step_upload(ctypes.byref(layout), ctypes.byref(step.c), ctypes.byref(pool), wp, wb,
                                     _stream(stream), ctypes.byref(plan)))
    plan._workspace = workspace
    plan._like = like
    return plan


def _rows(what: str, x, stride: Optional[int], n: int, width: int, like: Optional[_Like]):
    """(address, elements between tokens) of n rows: a tensor, a row a token and each row packed, or an address.
    A tensor of one row has no stride (0: packed). With a stride given, a tensor is where the rows begin."""
    if x is None or isinstance(x, int):
        return x, 0 if stride is None else stride
    if like is None:
        return x.data_ptr(), (x.stride(0) if x.size(0) > 1 else 0) if stride is None else stride
    shape, strides, fits = x.shape, x.stride(), True
    if stride is None:
        have = 1  # elements of a token, if they follow one another
        if len(shape) == 2:  # (the usual case)
            have = shape[1]
            fits = strides[1] == 1 or have == 1
        else:
            for d in range(len(shape) - 1, 0, -1):
                if strides[d] != have and shape[d] != 1:
                    fits = False
                have *= shape[d]
        stride = strides[0] if shape and shape[0] > 1 else 0
        # (a stride of 0, one row for all tokens, would mean packed to the library)
        if n and (not shape or shape[0] < n or have < width or (stride == 0 and n > 1)):
            fits = False
    elif n and stride >= 0:
        reach = x.storage_offset() + (stride or width) * (n - 1) + width
        fits = reach * x.element_size() <= x.untyped_storage().nbytes()
    if not fits or x.dtype is not like.dtype:
        raise ValueError(f"{what}: {tuple(shape)} of {x.dtype}, strides {strides}; {n} rows of {width} packed elements of {like.dtype} are needed")
    if not x.is_cuda:
        _on_gpu(what, x)
    return x.data_ptr(), stride


def append(plan: Plan, layer: int, *, k, v=None, q=None, q_out=None, q_weight=None, k_weight=None, eps: float = 1e-6,
           q_stride: Optional[int] = None, k_stride: Optional[int] = None, v_stride: Optional[int] = None,
           q_out_stride: Optional[int] = None, stream=None) -> None:
    """Norm and rotate the step's queries and keys; write its K and V rows into layer `layer`."""
    n, like = plan.num_tokens, plan._like
    wq = wk = 0
    if like is not None:
        wq, wk = like.q, like.k
        q_weight = _flat("q_weight", q_weight, like.dtype, like.dk, True)
        k_weight = _flat("k_weight", k_weight, like.dtype, like.normed, True)
    qp, qs = _rows("q", q, q_stride, n, wq, like)
    kp, ks = _rows("k", k, k_stride, n, wk, like)
    vp, vs = _rows("v", v, v_stride, n, wk, like if like is not None and like.gqa else None)  # (MLA: not read)
    op, os_ = _rows("q_out", q_out, q_out_stride, n, wq, like)
    rows = AppendRows(qp, kp, vp, op, qs, ks, vs, os_, _ptr(q_weight), _ptr(k_weight), eps, 0)
    status = (_bound or _lib()).kamera_step_append(ctypes.byref(plan), layer, ctypes.byref(rows), _stream(stream))
    if status:
        _check(status)


def attend(plan: Plan, layer: int, q, out, scale: float, lse=None, *, q_stride: Optional[int] = None,
           out_stride: Optional[int] = None, stream=None) -> None:
    """Attention of the step's query tokens over layer `layer` of the pool."""
    n, like = plan.num_tokens, plan._like
    wq = wo = 0
    if like is not None:
        wq, wo = like.q, like.out
        lse = _flat("lse", lse, like.stats, n * like.heads)
    qp, qs = _rows("q", q, q_stride, n, wq, like)
    op, os_ = _rows("out", out, out_stride, n, wo, like)
    status = (_bound or _lib()).kamera_step_attend(ctypes.byref(plan), layer, qp, qs, op, os_, _ptr(lse), scale, _stream(stream))
    if status:
        _check(status)


def copy_pages_workspace_bytes(num_copies: int) -> int:
    return int(_lib().kamera_copy_pages_workspace_bytes(int(num_copies)))


def _page_ids(x) -> np.ndarray:
    """Page ids as contiguous int32; ids that int32 does not hold are refused, not wrapped into others."""
    a = np.asarray(x)
    if a.size and a.dtype.kind not in "iu":
        raise ValueError(f"page ids are whole numbers, not {a.dtype}")
    ids = np.ascontiguousarray(a, dtype=np.int32)
    if a.dtype != np.int32 and (ids != a).any():
        raise ValueError("a page id does not fit 32 bits")
    return ids


def copy_pages(layout: Layout, pool: Pool, src, dst, workspace, stream=None) -> None:
    """Page dst[i] becomes what page src[i] was, for all i at once, in every layer."""
    s, d = _page_ids(src), _page_ids(dst)
    if s.shape != d.shape or s.ndim != 1:
        raise ValueError("src and dst are one-dimensional and of one length")
    wp, wb = _ws(workspace)
    _check(_lib().kamera_copy_pages(ctypes.byref(layout), ctypes.byref(pool), s.ctypes.data, d.ctypes.data, s.size, wp, wb,
                                    _stream(stream)))


def compact_pages(layout: Layout, pool: Pool, tables: Sequence[np.ndarray], workspace, stream=None) -> int:
    """Move the pages that `tables` (int32 host arrays, rewritten in place) name to the pool's start; their number."""
    for t in tables:
        if t.dtype != np.int32 or not t.flags.c_contiguous or not t.flags.writeable:
            raise ValueError("tables are writable, contiguous int32 arrays")
    n = len(tables)
    ptrs = (ctypes.c_void_p * max(n, 1))(*[t.ctypes.data for t in tables])
    lengths = np.array([t.size for t in tables] or [0], dtype=np.int32)
    live = ctypes.c_int32()
    wp, wb = _ws(workspace)
    _check(_lib().kamera_compact_pages(ctypes.byref(layout), ctypes.byref(pool), ptrs, lengths.ctypes.data, n,
                                       ctypes.byref(live), wp, wb, _stream(stream)))
    return int(live.value)
