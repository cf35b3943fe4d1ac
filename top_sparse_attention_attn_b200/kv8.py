"""Serving over a paged KV cache held in 8 bits: the PyTorch-facing wrapper of
`sa_page_plan`, `sa_kv8_write` and `sa_kv8_fwd`.

A serving step runs the three in this order:

    plan = plan_pages(lens, new_lens, block_table, free_pages, n_free, page_size=64, n_tokens=T)
    cache.write(k, v, block_table, plan.seq_lens, cu_seqlens_q=plan.cu_seqlens_q)
    o, lse = cache.attend(q, block_table, plan.seq_lens, cu_seqlens_q=plan.cu_seqlens_q)

`plan.slots` names the same rows for a 16-bit cache (rows of `SparseAttention`'s paged
k / v), whose writer is an index_copy.  Nothing here synchronises; the calls capture into
CUDA graphs.  Marshalling and checks only: all computation happens in the kernels.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib as L
from .api import _ELEMENT_TYPES

_FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_CODES = {torch.float8_e4m3fn: L.SA_KV8_E4M3, torch.int8: L.SA_KV8_INT8}


class PagePlan(NamedTuple):
    seq_lens: torch.Tensor       # [B] int32: rows of each request, its new tokens included
    cu_seqlens_q: torch.Tensor   # [B + 1] int32: offsets of the served requests' tokens
    slots: torch.Tensor          # [n_tokens] int64: cache row of each token, -1 = none
    n_free: torch.Tensor         # [1] int32: free pages left on the stack
    n_served: torch.Tensor       # [1] int32: requests served (the first ones)


# A decode step's calls take a few microseconds on the GPU, so the checks below are kept to a
# few attribute reads per tensor; what is wrong is worked out only once something is.

_INT32, _FP32 = torch.int32, torch.float32


def _refuse(t, name, dtype, index, shape):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} is {getattr(t, 'dtype', type(t))}: {dtype} expected")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}: device {index} expected")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}: {tuple(shape)} expected")
    raise ValueError(f"{name} is not contiguous")


def _vec(t, name, n, index):
    """Pointer of a contiguous int32 [n]."""
    if t.dtype is not _INT32 or t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        _refuse(t, name, _INT32, index, (n,))
    return t.data_ptr()


def _need(t, name, dtype, index, shape):
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dtype, index, shape)
    return t.data_ptr()


def _table(t, index):
    """(pointer, B, max_pages, elements from row to row) of a block table whose rows are contiguous."""
    if t.dtype is not _INT32 or t.dim() != 2:
        raise TypeError(f"block_table is {t.dtype} with {t.dim()} axes: int32 [B, max_pages] expected")
    if t.get_device() != index:
        raise ValueError(f"block_table is on {t.device}: device {index} expected")
    (B, n), (row, col) = t.shape, t.stride()
    if n > 1 and col != 1:
        raise ValueError("block_table rows are not contiguous")
    return t.data_ptr(), B, n, row if row > n else n


def _rows(t, name, heads, d, index):
    """(pointer, elements from token to token) of [T, heads, d] or [B, s, heads, d] whose
    tokens lie evenly apart and whose token rows are contiguous."""
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}: device {index} expected")
    shape, st = t.shape, t.stride()
    if len(shape) not in (3, 4) or shape[-2] != heads or shape[-1] != d:
        raise ValueError(f"{name} has shape {tuple(shape)}: [T, {heads}, {d}] or [B, s, {heads}, {d}] expected")
    if (st[-1] != 1 and d > 1) or (heads > 1 and st[-2] != d):
        raise ValueError(f"{name}: a token's row [{heads}, {d}] is not contiguous")
    if len(shape) == 3:
        step = st[0] if shape[0] > 1 else heads * d
    elif shape[1] > 1:
        step = st[1]
        if shape[0] > 1 and st[0] != step * shape[1]:
            raise ValueError(f"{name}: tokens do not lie evenly apart")
    else:
        step = st[0] if shape[0] > 1 else heads * d
    return t.data_ptr(), step


def _launch(fn, where, index, stream, *args):
    """Calls fn(*args, stream) with device `index` current, on its current stream unless one is given."""
    if index < 0:
        raise ValueError("the tensors are on the CPU: a CUDA device expected")
    before = torch.cuda.current_device()
    if before != index:
        torch.cuda.set_device(index)
    try:
        status = fn(*args, torch.cuda.current_stream(index).cuda_stream if stream is None else stream)
    finally:
        if before != index:
            torch.cuda.set_device(before)
    if status:
        raise L.SaError(status, where)


def plan_pages(old_lens, new_lens, block_table, free_pages, n_free, *, page_size: int, n_tokens: int,
               stream=None) -> PagePlan:
    """The page plan of a serving step (sa_page_plan).

    old_lens, new_lens [B] int32; block_table [B, max_pages] int32, updated in place (the
    first ceil(old / page_size) entries of a row are its pages); free_pages int32, a stack of
    which the first n_free[0] (int32 [1]) are free, taken from the end; n_tokens: the packed
    token axis.  Requests are served in order up to the first that does not fit."""
    index = old_lens.get_device()
    B = old_lens.shape[0] if old_lens.dim() == 1 else -1
    if B < 0 or free_pages.dim() != 1:
        raise ValueError("old_lens [B] and free_pages [n] expected")
    a = L.SaPagePlanArgs()
    a.batch, a.page_size, a.n_tokens = B, page_size, n_tokens
    a.old_lens = _vec(old_lens, "old_lens", B, index)
    a.new_lens = _vec(new_lens, "new_lens", B, index)
    n = a.free_capacity = free_pages.shape[0]
    a.free_pages = _vec(free_pages, "free_pages", n, index)
    a.n_free = _vec(n_free, "n_free", 1, index)
    a.block_table, rows, a.max_pages, a.table_stride = _table(block_table, index)
    if rows != B:
        raise ValueError(f"block_table has {rows} rows: {B} expected")
    lens, cu, left, served = (old_lens.new_empty(n) for n in (B, B + 1, 1, 1))
    slots = old_lens.new_empty(n_tokens if n_tokens > 0 else 0, dtype=torch.int64)
    a.seq_lens, a.cu_seqlens_q, a.slots = lens.data_ptr(), cu.data_ptr(), slots.data_ptr()
    a.n_free_out, a.n_served = left.data_ptr(), served.data_ptr()
    _launch(L.lib().sa_page_plan, "sa_page_plan", index, stream, ctypes.byref(a))
    return PagePlan(lens, cu, slots, left, served)


class Kv8Cache:
    """A paged KV cache held in 8 bits, one scale per page and head (see sa_kv8_cache).

    k [n_pages, page_size, Hkv, d_qk] and v [n_pages, page_size, Hkv, d_v] are codes
    (torch.float8_e4m3fn or torch.int8), k_scale and v_scale [n_pages, Hkv] fp32.  Without v
    the row is shared: V is its first d_v columns."""

    def __init__(self, k, v, k_scale, v_scale, *, d_v: int | None = None):
        if k.dtype not in _CODES:
            raise TypeError(f"k is {k.dtype}: float8_e4m3fn or int8 expected")
        if k.dim() != 4:
            raise ValueError("k is [n_pages, page_size, Hkv, d_qk]")
        P, ps, H, d = (int(x) for x in k.shape)
        index = k.get_device()
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads_kv, self.d_qk = P, ps, H, d
        self.d_v = int(v.shape[-1]) if v is not None else int(d if d_v is None else d_v)
        if d_v is not None and self.d_v != d_v:
            raise ValueError(f"v has {self.d_v} columns: {d_v} expected")
        self.device, self._index = k.device, index
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)  # bits of sa_kv8_cache.status
        c = L.SaKv8Cache()
        c.format = _CODES[k.dtype]
        c.n_heads_kv, c.d_qk, c.d_v, c.kv_shared = H, d, self.d_v, 1 if v is None else 0
        c.page_size, c.n_pages = ps, P
        c.k = _need(k, "k", k.dtype, index, (P, ps, H, d))
        c.k_scale = _need(k_scale, "k_scale", _FP32, index, (P, H))
        if v is not None:
            c.v = _need(v, "v", k.dtype, index, (P, ps, H, self.d_v))
            c.v_scale = _need(v_scale, "v_scale", _FP32, index, (P, H))
        c.status = self.status.data_ptr()
        self._c = c

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_heads_kv: int, d_qk: int, d_v: int, *, shared: bool = False,
              fmt: str = "e4m3", device="cuda") -> "Kv8Cache":
        """A cache of zero codes."""
        dt = _FORMATS[fmt]
        k = torch.zeros((n_pages, page_size, n_heads_kv, d_qk), dtype=torch.int8, device=device).view(dt)
        ks = torch.zeros((n_pages, n_heads_kv), dtype=torch.float32, device=device)
        if shared:
            return cls(k, None, ks, None, d_v=d_v)
        v = torch.zeros((n_pages, page_size, n_heads_kv, d_v), dtype=torch.int8, device=device).view(dt)
        return cls(k, v, ks, torch.zeros_like(ks), d_v=d_v)

    def _step(self, x, name, block_table, seq_lens, cu_seqlens_q):
        """The cache's description for the tokens of x ([T, ..] with offsets, or [B, s, ..])."""
        index = self._index
        c = L.SaKv8Cache.from_buffer_copy(self._c)
        c.block_table, B, c.max_pages, c.table_stride = _table(block_table, index)
        c.batch = B
        c.seq_lens = _vec(seq_lens, "seq_lens", B, index)
        if cu_seqlens_q is not None:
            if x.dim() != 3:
                raise ValueError(f"{name} is [T, heads, d] where cu_seqlens_q is given")
            c.layout, c.t_q = L.SA_LAYOUT_TND, x.shape[0]
            c.cu_seqlens_q = _vec(cu_seqlens_q, "cu_seqlens_q", B + 1, index)
        else:
            if x.dim() != 4 or x.shape[0] != B:
                raise ValueError(f"{name} is [B, s, heads, d] where cu_seqlens_q is not given")
            c.layout, c.s_q = L.SA_LAYOUT_BSND, x.shape[1]
        return c

    def write(self, k, v, block_table, seq_lens, *, cu_seqlens_q=None, stream=None) -> None:
        """Round the step's rows to 8 bits into their pages (sa_kv8_write).

        k [T, Hkv, d_qk] (or [B, s, Hkv, d_qk]) and v likewise, bfloat16 or float16, are the
        last rows of their sequences; seq_lens counts them.  The pages' scales grow where the
        rows need it.  v is None for a shared row."""
        if k.dtype not in _ELEMENT_TYPES:
            raise TypeError(f"k is {k.dtype}: bfloat16 or float16 expected")
        if (v is None) != (self.v is None):
            raise ValueError("v goes with a cache of separate K and V")
        c = self._step(k, "k", block_table, seq_lens, cu_seqlens_q)
        r = L.SaKv8Rows()
        r.dtype = _ELEMENT_TYPES[k.dtype]
        r.k, r.k_stride = _rows(k, "k", self.n_heads_kv, self.d_qk, self._index)
        if v is not None:
            if v.dtype != k.dtype or v.shape[:-1] != k.shape[:-1]:
                raise TypeError(f"v is {v.dtype} {tuple(v.shape)}, k is {k.dtype} {tuple(k.shape)}")
            r.v, r.v_stride = _rows(v, "v", self.n_heads_kv, self.d_v, self._index)
        _launch(L.lib().sa_kv8_write, "sa_kv8_write", self._index, stream, ctypes.byref(c), ctypes.byref(r))

    def attend(self, q, block_table, seq_lens, *, cu_seqlens_q=None, idx=None, block_size: int = 1, topk_len=None,
               window: int | None = None, sinks=None, scale: float | None = None, o=None, lse=None, stream=None):
        """Attention of the step's query tokens over the cache (sa_kv8_fwd): (o, lse).

        q [T, Hq, d_qk] (or [B, s, Hq, d_qk]): the last tokens of their sequences, each seeing
        the rows up to its own, of them the last window + 1 if window is given, and of those
        the ones its indices select if idx [.., Hkv, topk] is given (blocks of block_size
        rows).  sinks [Hq] fp32.  scale defaults to d_qk ** -0.5.  o and lse may be given; rows
        behind the last sequence stay as they are."""
        if q.dtype not in _ELEMENT_TYPES:
            raise TypeError(f"q is {q.dtype}: bfloat16 or float16 expected")
        index, H = self._index, self.n_heads_kv
        c = self._step(q, "q", block_table, seq_lens, cu_seqlens_q)
        shape = q.shape
        lead, Hq = shape[:-2], shape[-2]
        a = L.SaKv8Query()
        a.dtype = _ELEMENT_TYPES[q.dtype]
        a.n_heads_q, a.block_size = Hq, block_size
        if window is None:
            a.win_left = -1
        elif window < 0:
            raise ValueError("window is the rows before a token's own that it sees: 0 or more")
        else:
            a.win_left = window
        a.scale = self.d_qk ** -0.5 if scale is None else scale
        a.q, a.q_stride = _rows(q, "q", Hq, self.d_qk, index)
        if idx is not None:
            topk = idx.shape[-1]
            if topk == 0:
                raise ValueError("idx has no slots")
            a.idx, a.topk = _need(idx, "idx", _INT32, index, (*lead, H, topk)), topk
            if topk_len is not None:
                a.topk_len = _need(topk_len, "topk_len", _INT32, index, (*lead, H))
        elif topk_len is not None:
            raise ValueError("topk_len goes with idx")
        if sinks is not None:
            a.sinks = _need(sinks, "sinks", _FP32, index, (Hq,))
        if o is None:
            o = q.new_empty((*lead, Hq, self.d_v))
            a.o = o.data_ptr()
        else:
            a.o = _need(o, "o", q.dtype, index, (*lead, Hq, self.d_v))
        if lse is None:
            lse = q.new_empty((*lead, Hq), dtype=_FP32)
            a.lse = lse.data_ptr()
        else:
            a.lse = _need(lse, "lse", _FP32, index, (*lead, Hq))
        pc, pa = ctypes.byref(c), ctypes.byref(a)
        lib, n = L.lib(), ctypes.c_size_t(0)
        status = lib.sa_kv8_fwd_get_workspace_size(pc, pa, ctypes.byref(n))
        if status:
            raise L.SaError(status, "sa_kv8_fwd_get_workspace_size")
        n = n.value
        ws = q.new_empty(n, dtype=torch.uint8)
        _launch(lib.sa_kv8_fwd, "sa_kv8_fwd", index, stream, pc, pa, ws.data_ptr(), n)
        return o, lse

    def read_status(self, stream=None) -> int:
        """The calls' status word so far, as an sa_status (synchronises the stream)."""
        with torch.cuda.device(self._index):
            st = torch.cuda.current_stream(self._index).cuda_stream if stream is None else stream
            return L.sa_read_status(self.status.data_ptr(), 4, st)

    def dequantize(self):
        """(k, v) as fp32 tensors of the cache's shape (v None for a shared row)."""
        k = self.k.float() * self.k_scale[:, None, :, None]
        return k, None if self.v is None else self.v.float() * self.v_scale[:, None, :, None]
