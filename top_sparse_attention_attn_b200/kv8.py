"""Serving over a paged KV cache held in 8 bits: the PyTorch-facing wrapper of
`sa_page_plan`, `sa_kv8_write` and `sa_kv8_fwd`.

A serving step runs the three in this order:

    plan = plan_pages(lens, new_lens, block_table, free_pages, n_free, page_size=64, n_tokens=T)
    cache.write(k, v, block_table, plan.seq_lens, cu_seqlens_q=plan.cu_seqlens_q)
    o, lse = cache.attend(q, block_table, plan.seq_lens, cu_seqlens_q=plan.cu_seqlens_q)

`plan.slots` names the same rows for a 16-bit cache (rows of `SparseAttention`'s paged
k / v), whose writer is an index_copy.  Nothing here synchronises; the calls capture into
CUDA graphs.  All computation happens in the kernels; tensors are checked and marshalled
by the module `_kv8_ext` (csrc/ext), which loading fails loudly without.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib as L

_FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_CODES = {torch.float8_e4m3fn: L.SA_KV8_E4M3, torch.int8: L.SA_KV8_INT8}


_module = None


def _ext():
    global _module
    if _module is None:
        from . import _kv8_ext
        _module = _kv8_ext
    return _module


class PagePlan(NamedTuple):
    seq_lens: torch.Tensor       # [B] int32: rows of each request, its new tokens included
    cu_seqlens_q: torch.Tensor   # [B + 1] int32: offsets of the served requests' tokens
    slots: torch.Tensor          # [n_tokens] int64: cache row of each token, -1 = none
    n_free: torch.Tensor         # [1] int32: free pages left on the stack
    n_served: torch.Tensor       # [1] int32: requests served (the first ones)


def _check(r, where):
    if type(r) is int and r != L.SA_OK:
        raise L.SaError(r, where)
    return r


def plan_pages(old_lens, new_lens, block_table, free_pages, n_free, *, page_size: int, n_tokens: int,
               stream=None) -> PagePlan:
    """The page plan of a serving step (sa_page_plan).

    old_lens, new_lens [B] int32; block_table [B, max_pages] int32, updated in place (the
    first ceil(old / page_size) entries of a row are its pages); free_pages int32, a stack of
    which the first n_free[0] (int32 [1]) are free, taken from the end; n_tokens: the packed
    token axis.  Requests are served in order up to the first that does not fit."""
    r = _ext().plan(old_lens, new_lens, block_table, free_pages, n_free, page_size, n_tokens, stream)
    return PagePlan(*_check(r, "sa_page_plan"))


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
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads_kv, self.d_qk = P, ps, H, d
        self.d_v = int(v.shape[-1]) if v is not None else int(d if d_v is None else d_v)
        if d_v is not None and self.d_v != d_v:
            raise ValueError(f"v has {self.d_v} columns: {d_v} expected")
        self.device, self._index = k.device, k.get_device()
        self._scale = d ** -0.5
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)  # bits of sa_kv8_cache.status
        c = L.SaKv8Cache()
        c.format = _CODES[k.dtype]
        c.n_heads_kv, c.d_qk, c.d_v, c.kv_shared = H, d, self.d_v, 1 if v is None else 0
        c.page_size, c.n_pages = ps, P
        c.k = self._need(k, "k", k.dtype, (P, ps, H, d))
        c.k_scale = self._need(k_scale, "k_scale", torch.float32, (P, H))
        if v is not None:
            c.v = self._need(v, "v", k.dtype, (P, ps, H, self.d_v))
            c.v_scale = self._need(v_scale, "v_scale", torch.float32, (P, H))
        c.status = self.status.data_ptr()
        self._c = bytes(c)  # the description that each call completes with its tokens

    def _need(self, t, name, dtype, shape):
        if t is None or t.dtype != dtype:
            raise TypeError(f"{name} is {None if t is None else t.dtype}: {dtype} expected")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}: {self.device} expected")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}: {shape} expected")
        if not t.is_contiguous():
            raise ValueError(f"{name} is not contiguous")
        return t.data_ptr()

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

    def write(self, k, v, block_table, seq_lens, *, cu_seqlens_q=None, stream=None) -> None:
        """Round the step's rows to 8 bits into their pages (sa_kv8_write).

        k [T, Hkv, d_qk] (or [B, s, Hkv, d_qk]) and v likewise, bfloat16 or float16, are the
        last rows of their sequences; seq_lens counts them.  The pages' scales grow where the
        rows need it.  v is None for a shared row."""
        _check(_ext().write(self._c, self._index, k, v, block_table, seq_lens, cu_seqlens_q, stream), "sa_kv8_write")

    def attend(self, q, block_table, seq_lens, *, cu_seqlens_q=None, idx=None, block_size: int = 1, topk_len=None,
               window: int | None = None, sinks=None, scale: float | None = None, o=None, lse=None, stream=None):
        """Attention of the step's query tokens over the cache (sa_kv8_fwd): (o, lse).

        q [T, Hq, d_qk] (or [B, s, Hq, d_qk]): the last tokens of their sequences, each seeing
        the rows up to its own, of them the last window + 1 if window is given, and of those
        the ones its indices select if idx [.., Hkv, topk] is given (blocks of block_size
        rows).  sinks [Hq] fp32.  scale defaults to d_qk ** -0.5.  o and lse may be given; rows
        behind the last sequence stay as they are."""
        r = _ext().attend(self._c, self._index, q, block_table, seq_lens, cu_seqlens_q, idx, block_size, topk_len, window,
                          sinks, self._scale if scale is None else scale, o, lse, stream)
        return _check(r, "sa_kv8_fwd")

    def read_status(self, stream=None) -> int:
        """The calls' status word since it was last cleared, as an sa_status (synchronises the stream)."""
        with torch.cuda.device(self._index):
            st = torch.cuda.current_stream(self._index).cuda_stream if stream is None else stream
            return L.sa_read_status(self.status.data_ptr(), 4, st)

    def clear_status(self, stream=None) -> None:
        """Clear the status word, in the stream's order: what read_status reported is not reported again, and
        the calls behind it no longer give up their waits for a time-out that was met before."""
        if self._index < 0 or stream is None:
            self.status.zero_()
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device)):
                self.status.zero_()

    def dequantize(self):
        """(k, v) as fp32 tensors of the cache's shape (v None for a shared row), as attend reads them."""
        def values(codes, scale):
            s = torch.where(scale.isnan(), 0.0, scale).clamp(2.0 ** -60, 2.0 ** 60)
            return codes.float() * s[:, None, :, None]
        return values(self.k, self.k_scale), None if self.v is None else values(self.v, self.v_scale)
