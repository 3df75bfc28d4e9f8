"""A torch-facing handle on a paged K/V cache: argument marshalling over ``ibp``.

The cache holds the keys and values of many sequences in pages of
``page_tokens`` tokens; a ``PagedBatch`` names the sequences of one step (their
pages, lengths and new tokens).  Every call goes straight to the C-ABI library;
this class checks shapes and types, allocates outputs and passes pointers.

    cache = PagedCache(kv_heads=8, head_dim=128, page_tokens=16, n_pages=4096)
    batch = cache.batch(page_table, kv_lens, q_starts, n_tokens, max_q_tokens)
    q = cache.append(batch, k, v, q=q, q_norm=qw, k_norm=kw, cos_sin=table)
    out = cache.attention(batch, q)                       # over every cached token

    cache.update_bounds(batch, bounds)                    # or over the pages that score best
    pages = cache.select_pages(batch, cache.page_scores(batch, q, bounds), 64)
    out = cache.attention(batch, q, pages=pages)

A token's keys (or values) over all heads are one row of ``kv_heads *
head_dim`` 16-bit values, so pages go to a compressed host store and come back
through ``IbpStore``: ``key_rows()`` and ``value_rows()`` are the rows.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple, Union

import torch

from . import ibp

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
# the current stream's handle, by device (a torch without CUDA has none)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# Attention's workspace of each (device, stream): calls on one stream follow one another
# there, and the library enqueues those of several threads one after the other.
_workspaces = {}


def _workspace(device: torch.device, raw: int) -> torch.Tensor:
    if torch._C._cuda_isCurrentStreamCapturing():  # a graph's replays may run on any stream
        return torch.empty(ibp.PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
    ws = _workspaces.get((device.index, raw))
    if ws is None:
        ws = _workspaces.setdefault((device.index, raw), torch.empty(
            ibp.PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=device))
    return ws


def _as_stream(stream) -> torch.cuda.Stream:
    if not isinstance(stream, int):
        return stream
    # (an ExternalStream of 0 is a new stream, not the default one)
    return torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()


class PagedBatch:
    """The sequences of one step; keeps its tensors alive."""

    __slots__ = ("desc", "address", "page_table", "kv_lens", "q_starts", "n_tokens", "max_pages",
                 "index")

    def __init__(self, page_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor,
                 n_tokens: int, max_q_tokens: int):
        n = kv_lens.numel()
        for name, t in (("page_table", page_table), ("kv_lens", kv_lens), ("q_starts", q_starts)):
            if t.dtype != torch.int32 or not t.is_cuda:
                raise ValueError("%s must be an int32 device tensor" % name)
        self.index = kv_lens.get_device()
        if page_table.get_device() != self.index or q_starts.get_device() != self.index:
            raise ValueError("page_table, kv_lens and q_starts must be on one device")
        if (page_table.dim() != 2 or page_table.shape[0] != n or q_starts.numel() != n + 1
                or not kv_lens.is_contiguous() or not q_starts.is_contiguous()
                or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
            raise ValueError("page_table [n, pages], kv_lens [n] and q_starts [n + 1], contiguous")
        self.page_table, self.kv_lens, self.q_starts = page_table, kv_lens, q_starts
        self.n_tokens, self.max_pages = int(n_tokens), page_table.shape[1]
        stride = page_table.stride(0) if n > 1 else max(page_table.stride(0), self.max_pages)
        self.desc = ibp.ibp_paged_batch(page_table.data_ptr(), kv_lens.data_ptr(),
                                        q_starts.data_ptr(), stride, n, self.max_pages,
                                        self.n_tokens, int(max_q_tokens))
        self.address = ctypes.addressof(self.desc)


class PagedCache:
    """Key and value pages of one layer, [n_pages, page_tokens, kv_heads, head_dim]
    (any strides of whole heads; allocated when not given).

    Calls run on the current stream, or on `stream` (a torch stream or a
    cudaStream_t), on which their outputs and workspaces are then allocated too.
    The pages' device has to be the current one.  Several threads may call on one
    stream.  The operators are for serving: results carry no gradient, also where
    the arguments require one."""

    def __init__(self, kv_heads: int, head_dim: int, page_tokens: int, n_pages: int,
                 dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None,
                 v: Optional[torch.Tensor] = None, device=None):
        self.handle = None
        if dtype not in _DTYPES:
            raise ValueError("a paged cache holds float16 or bfloat16")
        shape = (n_pages, page_tokens, kv_heads, head_dim)
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        if k is None:
            device = device or torch.device("cuda", torch.cuda.current_device())
            k = torch.empty(shape, dtype=dtype, device=device)
            v = torch.empty(shape, dtype=dtype, device=device)
        for t in (k, v):
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_cuda or t.stride(3) != 1:
                raise ValueError("k and v must be device tensors [n_pages, page_tokens, kv_heads, "
                                 "head_dim] of the cache's type, each head contiguous")
        if k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must have the same strides and device")
        self.kv_heads, self.head_dim, self.page_tokens = kv_heads, head_dim, page_tokens
        self.n_pages, self.dtype, self.k, self.v = n_pages, dtype, k, v
        self.device, self._index = k.device, k.device.index
        self._bounds_shape = (n_pages, kv_heads, 2, head_dim)
        # a dimension of one element has no stride to speak of
        row = head_dim * 2
        st = [s * 2 if n > 1 else max(s * 2, row) for s, n in zip(k.stride(), shape)]
        self._lib = ibp._lib_handle()
        with torch.cuda.device(self._index):  # the handle belongs to the pages' device
            self.handle = ibp.ibp_paged_create(ibp.ibp_paged_desc(
                k.data_ptr(), v.data_ptr(), st[0], st[2], st[1], n_pages, page_tokens, kv_heads,
                head_dim, _DTYPES[dtype]))

    # -- lifetime
    def close(self) -> None:
        if self.handle:
            ibp.ibp_paged_destroy(self.handle)
            self.handle = None

    def __enter__(self) -> "PagedCache":
        return self

    def __exit__(self, *exc) -> None:
        self.close()

    def __del__(self) -> None:
        try:
            self.close()
        except Exception:  # the interpreter or the context is going away
            pass

    def status(self, stream=None, reset: bool = True) -> int:
        """The device status word (synchronises the stream)."""
        return ibp.ibp_paged_status(self.handle, stream, reset)

    # -- rows for a compressed store
    def _rows(self, t: torch.Tensor) -> torch.Tensor:
        n = self.n_pages * self.page_tokens
        return t.view(n, self.kv_heads * self.head_dim).view(torch.uint8)

    def key_rows(self) -> torch.Tensor:
        """The keys as bytes [n_pages * page_tokens, row_bytes] (contiguous pages)."""
        return self._rows(self.k)

    def value_rows(self) -> torch.Tensor:
        return self._rows(self.v)

    # -- calls
    # Tensors that are not on the cache's device are refused: a kernel would take their
    # addresses for this device's.
    def batch(self, page_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor,
              n_tokens: int, max_q_tokens: int) -> PagedBatch:
        """A step's sequences: page_table [n, pages], kv_lens [n] (tokens in the
        cache, the new ones among them), q_starts [n + 1] (rows of each sequence's
        new tokens), int32 on the device; n_tokens rows in all, of one sequence at
        most max_q_tokens."""
        return PagedBatch(page_table, kv_lens, q_starts, n_tokens, max_q_tokens)

    def _heads(self, name: str, t: torch.Tensor, batch: PagedBatch, heads: Optional[int]) -> int:
        """Checks a [n_tokens, heads, head_dim] tensor; its token stride in bytes."""
        s, st = t.shape, t.stride()
        if (batch.index != self._index or len(s) != 3 or s[0] != batch.n_tokens
                or s[2] != self.head_dim or t.dtype is not self.dtype
                or t.get_device() != self._index or st[2] != 1
                or (heads is not None and s[1] != heads) or (s[1] > 1 and st[1] != s[2])):
            raise ValueError("%s must be a tensor [n_tokens, heads, head_dim] of the cache's type "
                             "and device (as the batch) whose heads lie side by side" % name)
        return st[0] * 2 if s[0] > 1 else s[1] * s[2] * 2

    def append(self, batch: PagedBatch, k: torch.Tensor, v: torch.Tensor,
               q: Optional[torch.Tensor] = None, q_norm: Optional[torch.Tensor] = None,
               k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
               cos_sin: Optional[torch.Tensor] = None, pairs: bool = False,
               q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
        """Writes k and v [n_tokens, kv_heads, head_dim] into their pages; k and q
        normalised for each head (weights q_norm, k_norm) and rotated (cos_sin fp32
        [positions, rot_dim]: cosines, then sines) on the way.  Returns the queries."""
        if stream is not None:
            with torch.cuda.stream(_as_stream(stream)):
                return self.append(batch, k, v, q, q_norm, k_norm, eps, cos_sin, pairs, q_out)
        ks = self._heads("k", k, batch, self.kv_heads)
        if self._heads("v", v, batch, self.kv_heads) != ks:
            raise ValueError("k and v must have the same token stride")
        qs = os = heads = 0
        if q is not None:
            qs = self._heads("q", q, batch, None)
            heads = q.shape[1]
            if heads == 0:
                raise ValueError("q has no heads")
            if q_out is None:
                q_out = torch.empty((batch.n_tokens, heads, self.head_dim), dtype=q.dtype,
                                    device=q.device)
                os = heads * self.head_dim * 2
            else:
                os = self._heads("q_out", q_out, batch, heads)
        for name, w in ((("q_norm", q_norm), ("k_norm", k_norm))
                        if q_norm is not None or k_norm is not None else ()):
            if w is not None and (w.shape != (self.head_dim,) or w.dtype != self.dtype
                                  or w.get_device() != self._index or not w.is_contiguous()):
                raise ValueError("%s must be [head_dim] of the cache's type and device" % name)
        n_pos = rot = 0
        if cos_sin is not None:
            if (cos_sin.dim() != 2 or cos_sin.dtype != torch.float32
                    or cos_sin.get_device() != self._index or not cos_sin.is_contiguous()):
                raise ValueError("cos_sin must be a contiguous float32 [positions, rot_dim] on "
                                 "the cache's device")
            n_pos, rot = cos_sin.shape
            if n_pos == 0 or rot == 0:  # its null pointer would say that there is none
                raise ValueError("cos_sin has no elements")
        ibp._check(self._lib.ibp_paged_append(
            self.handle, batch.address, k.data_ptr(), v.data_ptr(), ks,
            None if q is None else q.data_ptr(), qs, None if q is None else q_out.data_ptr(), os,
            heads, None if q_norm is None else q_norm.data_ptr(),
            None if k_norm is None else k_norm.data_ptr(), eps,
            None if cos_sin is None else cos_sin.data_ptr(), n_pos, rot, 1 if pairs else 0,
            _raw_stream(self._index)), "ibp_paged_append")
        return q_out

    def attention(self, batch: PagedBatch, q: torch.Tensor, scale: Optional[float] = None,
                  causal: bool = True, window: int = 0, pages: Optional[torch.Tensor] = None,
                  lse: bool = False, out: Optional[torch.Tensor] = None, stream=None
                  ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
        """Attention of q [n_tokens, q_heads, head_dim] over the cached tokens, or
        over the selected pages (int32 [n_tokens, kv_heads, n]); with lse=True also
        the log of each row's sum [n_tokens, q_heads].  scale: 1/sqrt(head_dim)."""
        if stream is not None:
            with torch.cuda.stream(_as_stream(stream)):
                return self.attention(batch, q, scale, causal, window, pages, lse, out)
        qs = self._heads("q", q, batch, None)
        heads = q.shape[1]
        if out is None:
            out = torch.empty((batch.n_tokens, heads, self.head_dim), dtype=q.dtype,
                              device=q.device)
        elif (out.get_device() != self._index or out.shape != q.shape or out.dtype != q.dtype
              or not out.is_contiguous()):
            raise ValueError("out must be contiguous, of q's shape, type and device")
        total = (torch.empty((batch.n_tokens, heads), dtype=torch.float32, device=q.device)
                 if lse else None)
        n = 0
        if pages is not None:
            if (pages.dim() != 3 or pages.shape[:2] != (batch.n_tokens, self.kv_heads)
                    or pages.dtype != torch.int32 or pages.get_device() != self._index
                    or not pages.is_contiguous()):
                raise ValueError("pages must be a contiguous int32 [n_tokens, kv_heads, n] on the "
                                 "cache's device")
            n = pages.shape[2]
            if n == 0:  # its null pointer would say that there are no lists
                raise ValueError("pages lists no pages")
        raw = _raw_stream(self._index)
        ws = _workspace(self.device, raw)
        ibp._check(self._lib.ibp_paged_attention(
            self.handle, batch.address, q.data_ptr(), qs, heads, out.data_ptr(),
            total.data_ptr() if lse else None,
            1.0 / math.sqrt(self.head_dim) if scale is None else scale, 1 if causal else 0, window,
            None if pages is None else pages.data_ptr(), n, ws.data_ptr(),
            ibp.PAGED_WORKSPACE_BYTES, raw), "ibp_paged_attention")
        return (out, total) if lse else out

    def _bounds(self, batch: PagedBatch, bounds: torch.Tensor) -> None:
        index = self._index
        if (batch.index != index or bounds.get_device() != index
                or bounds.shape != self._bounds_shape or bounds.dtype is not self.dtype
                or not bounds.is_contiguous()):
            raise ValueError("bounds must be a contiguous [n_pages, kv_heads, 2, head_dim] of the "
                             "cache's type and device (as the batch)")

    def update_bounds(self, batch: PagedBatch, bounds: torch.Tensor, stream=None) -> None:
        """Smallest and largest keys of the pages that the new tokens went into,
        into bounds [n_pages, kv_heads, 2, head_dim]."""
        if stream is not None:
            with torch.cuda.stream(_as_stream(stream)):
                return self.update_bounds(batch, bounds)
        self._bounds(batch, bounds)
        ibp._check(self._lib.ibp_paged_bounds(self.handle, batch.address, bounds.data_ptr(),
                                              _raw_stream(self._index)), "ibp_paged_bounds")

    def page_scores(self, batch: PagedBatch, q: torch.Tensor, bounds: torch.Tensor,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Upper bounds of q . k over each page, [n_tokens, kv_heads, max_pages]."""
        if stream is not None:
            with torch.cuda.stream(_as_stream(stream)):
                return self.page_scores(batch, q, bounds, out)
        self._bounds(batch, bounds)
        qs = self._heads("q", q, batch, None)
        shape = (batch.n_tokens, self.kv_heads, batch.max_pages)
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=q.device)
        elif (out.get_device() != self._index or out.shape != shape or out.dtype != torch.float32
              or not out.is_contiguous()):
            raise ValueError("out must be a contiguous float32 [n_tokens, kv_heads, max_pages] on "
                             "the cache's device")
        ibp._check(self._lib.ibp_paged_scores(
            self.handle, batch.address, q.data_ptr(), qs, q.shape[1], bounds.data_ptr(),
            out.data_ptr(), _raw_stream(self._index)), "ibp_paged_scores")
        return out

    def select_pages(self, batch: PagedBatch, scores: torch.Tensor, n: int,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The n pages of largest score of each token and head, int32
        [n_tokens, kv_heads, n], ascending, -1 behind the last."""
        if stream is not None:
            with torch.cuda.stream(_as_stream(stream)):
                return self.select_pages(batch, scores, n, out)
        if (batch.index != self._index
                or scores.shape != (batch.n_tokens, self.kv_heads, batch.max_pages)
                or scores.dtype != torch.float32 or scores.get_device() != self._index
                or not scores.is_contiguous()):
            raise ValueError("scores must be a contiguous float32 [n_tokens, kv_heads, max_pages] "
                             "on the cache's device (as the batch)")
        shape = (batch.n_tokens, self.kv_heads, n)
        if out is None:
            out = torch.empty(shape, dtype=torch.int32, device=scores.device)
        elif (out.get_device() != self._index or out.shape != shape or out.dtype != torch.int32
              or not out.is_contiguous()):
            raise ValueError("out must be a contiguous int32 [n_tokens, kv_heads, n] on the "
                             "cache's device")
        ibp._check(self._lib.ibp_paged_select(self.handle, batch.address, scores.data_ptr(), n,
                                              out.data_ptr(), _raw_stream(self._index)),
                   "ibp_paged_select")
        return out
