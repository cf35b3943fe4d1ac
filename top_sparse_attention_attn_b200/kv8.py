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


def _need(t, name, dtype, device, shape=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}: {dtype} expected")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}: {device} expected")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: {shape} expected")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return t.data_ptr()


def _table(t, device):
    if t.dtype != torch.int32 or t.dim() != 2:
        raise TypeError(f"block_table is {t.dtype} with {t.dim()} axes: int32 [B, max_pages] expected")
    if t.device != device:
        raise ValueError(f"block_table is on {t.device}: {device} expected")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("block_table rows are not contiguous")
    return t.data_ptr(), max(t.stride(0), t.shape[1])


def _rows(t, name, heads, d, device):
    """(pointer, elements from token to token) of [T, heads, d] or [B, s, heads, d] whose
    tokens lie evenly apart and whose token rows are contiguous."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}: {device} expected")
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


class _on:
    """Runs the block with `device` current, and gives its current stream unless one is given."""

    __slots__ = ("index", "before")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        self.before = self.index if self.index is None else torch.cuda.current_device()
        if self.index != self.before:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.index != self.before:
            torch.cuda.set_device(self.before)


def _stream(stream, device) -> int:
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}: a CUDA device expected")
    return torch.cuda.current_stream(device).cuda_stream if stream is None else stream


def plan_pages(old_lens, new_lens, block_table, free_pages, n_free, *, page_size: int, n_tokens: int,
               stream=None) -> PagePlan:
    """The page plan of a serving step (sa_page_plan).

    old_lens, new_lens [B] int32; block_table [B, max_pages] int32, updated in place (the
    first ceil(old / page_size) entries of a row are its pages); free_pages int32, a stack of
    which the first n_free[0] (int32 [1]) are free, taken from the end; n_tokens: the packed
    token axis.  Requests are served in order up to the first that does not fit."""
    dev = old_lens.device
    B = int(old_lens.numel())
    a = L.SaPagePlanArgs()
    a.batch, a.page_size, a.n_tokens = B, page_size, n_tokens
    a.old_lens = _need(old_lens, "old_lens", torch.int32, dev, (B,))
    a.new_lens = _need(new_lens, "new_lens", torch.int32, dev, (B,))
    if free_pages.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("free_pages [n] and block_table [B, max_pages] expected")
    a.free_pages = _need(free_pages, "free_pages", torch.int32, dev)
    a.free_capacity = int(free_pages.numel())
    a.n_free = _need(n_free, "n_free", torch.int32, dev, (1,))
    a.block_table, a.table_stride = _table(block_table, dev)
    a.max_pages = int(block_table.shape[1])
    out = torch.empty(2 * B + 3, dtype=torch.int32, device=dev)
    lens, cu, left, served = out[:B], out[B:2 * B + 1], out[2 * B + 1:2 * B + 2], out[2 * B + 2:]
    slots = torch.empty(max(n_tokens, 0), dtype=torch.int64, device=dev)
    base = out.data_ptr()
    a.seq_lens, a.cu_seqlens_q, a.n_free_out, a.n_served = base, base + 4 * B, base + 8 * B + 4, base + 8 * B + 8
    a.slots = slots.data_ptr()
    with _on(dev):
        L.sa_page_plan(a, _stream(stream, dev))
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
        dev = k.device
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads_kv, self.d_qk = P, ps, H, d
        self.d_v = int(v.shape[-1]) if v is not None else int(d if d_v is None else d_v)
        if d_v is not None and self.d_v != d_v:
            raise ValueError(f"v has {self.d_v} columns: {d_v} expected")
        self.device = dev
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)  # bits of sa_kv8_cache.status
        c = L.SaKv8Cache()
        c.format = _CODES[k.dtype]
        c.n_heads_kv, c.d_qk, c.d_v, c.kv_shared = H, d, self.d_v, 1 if v is None else 0
        c.page_size, c.n_pages = ps, P
        c.k = _need(k, "k", k.dtype, dev)
        c.k_scale = _need(k_scale, "k_scale", torch.float32, dev, (P, H))
        if v is not None:
            c.v = _need(v, "v", k.dtype, dev, (P, ps, H, self.d_v))
            c.v_scale = _need(v_scale, "v_scale", torch.float32, dev, (P, H))
        c.status = self.status.data_ptr()
        self._c = c
        self._ws_bytes = {}

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
        dev = self.device
        c = L.SaKv8Cache.from_buffer_copy(self._c)
        c.block_table, c.table_stride = _table(block_table, dev)
        B, c.max_pages = (int(n) for n in block_table.shape)
        c.batch = B
        c.seq_lens = _need(seq_lens, "seq_lens", torch.int32, dev, (B,))
        if cu_seqlens_q is not None:
            if x.dim() != 3:
                raise ValueError(f"{name} is [T, heads, d] where cu_seqlens_q is given")
            c.layout, c.t_q = L.SA_LAYOUT_TND, int(x.shape[0])
            c.cu_seqlens_q = _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, (B + 1,))
        else:
            if x.dim() != 4 or x.shape[0] != B:
                raise ValueError(f"{name} is [B, s, heads, d] where cu_seqlens_q is not given")
            c.layout, c.s_q = L.SA_LAYOUT_BSND, int(x.shape[1])
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
        r.k, r.k_stride = _rows(k, "k", self.n_heads_kv, self.d_qk, self.device)
        if v is not None:
            if v.dtype != k.dtype or v.shape[:-1] != k.shape[:-1]:
                raise TypeError(f"v is {v.dtype} {tuple(v.shape)}, k is {k.dtype} {tuple(k.shape)}")
            r.v, r.v_stride = _rows(v, "v", self.n_heads_kv, self.d_v, self.device)
        with _on(self.device):
            L.sa_kv8_write(c, r, _stream(stream, self.device))

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
        dev = self.device
        c = self._step(q, "q", block_table, seq_lens, cu_seqlens_q)
        Hq, lead = int(q.shape[-2]), q.shape[:-2]
        a = L.SaKv8Query()
        a.dtype = _ELEMENT_TYPES[q.dtype]
        a.n_heads_q, a.block_size = Hq, block_size
        a.win_left = -1 if window is None else window
        if window is not None and window < 0:
            raise ValueError("window is the rows before a token's own that it sees: 0 or more")
        a.scale = self.d_qk ** -0.5 if scale is None else scale
        a.q, a.q_stride = _rows(q, "q", Hq, self.d_qk, dev)
        topk = 0
        if idx is not None:
            topk = int(idx.shape[-1])
            if topk == 0:
                raise ValueError("idx has no slots")
            a.idx = _need(idx, "idx", torch.int32, dev, (*lead, self.n_heads_kv, topk))
            if topk_len is not None:
                a.topk_len = _need(topk_len, "topk_len", torch.int32, dev, (*lead, self.n_heads_kv))
        elif topk_len is not None:
            raise ValueError("topk_len goes with idx")
        a.topk = topk
        if sinks is not None:
            a.sinks = _need(sinks, "sinks", torch.float32, dev, (Hq,))
        if o is None:
            o = torch.empty((*lead, Hq, self.d_v), dtype=q.dtype, device=dev)
            a.o = o.data_ptr()
        else:
            a.o = _need(o, "o", q.dtype, dev, (*lead, Hq, self.d_v))
        if lse is None:
            lse = torch.empty((*lead, Hq), dtype=torch.float32, device=dev)
            a.lse = lse.data_ptr()
        else:
            a.lse = _need(lse, "lse", torch.float32, dev, (*lead, Hq))
        with _on(dev):
            # what a workspace takes follows from these sizes alone
            key = (lead, Hq, topk, block_size, window, c.max_pages, c.batch)
            n = self._ws_bytes.get(key)
            if n is None:
                n = self._ws_bytes[key] = L.sa_kv8_fwd_get_workspace_size(c, a)
            ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
            L.sa_kv8_fwd(c, a, ws.data_ptr() if n else None, n, _stream(stream, dev))
        return o, lse

    def read_status(self, stream=None) -> int:
        """The calls' status word so far, as an sa_status (synchronises the stream)."""
        with _on(self.device):
            return L.sa_read_status(self.status.data_ptr(), 4, _stream(stream, self.device))

    def dequantize(self):
        """(k, v) as fp32 tensors of the cache's shape (v None for a shared row)."""
        k = self.k.float() * self.k_scale[:, None, :, None]
        return k, None if self.v is None else self.v.float() * self.v_scale[:, None, :, None]
