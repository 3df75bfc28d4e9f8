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

With ``page_dtype=torch.float8_e4m3fn`` the pages hold one byte for each value, under a
scale for each page and head (``k_scales``, ``v_scales``: powers of two,
float8_e8m0fnu); every call is the same:

    cache = PagedCache(8, 128, 16, 4096, torch.bfloat16, page_dtype=torch.float8_e4m3fn)

The pages that sequences hold can be kept on the device:

    tables = cache.tables(n_seqs, max_pages)              # every page is free
    batch, slots = tables.resize(target, n_tokens, longest)  # lengths change: pages come and go
    cache.append(batch, k, v)                             # slots: the new tokens' rows
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple, Union

import torch

from . import ibp

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_CODES, _SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu
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


# Above this a call does without the larger workspace that chunks over 8-bit pages make use of.
_MOST_WORKSPACE = 2 << 30


def _large_workspace(device: torch.device, bytes_: int) -> torch.Tensor:
    """The call's alone: torch has it back, for what follows on the stream, when the call is
    enqueued (the 3 us that this takes are beside a kernel of hundreds)."""
    return torch.empty(bytes_, dtype=torch.uint8, device=device)


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
    (any strides of whole heads; allocated when not given).  `dtype` is the type of the
    calls' queries, keys, values and results, and of the pages unless `page_dtype` is
    float8_e4m3fn: then a page's keys (values) of one head are codes under the scale in
    k_scales (v_scales) [n_pages, kv_heads], float8_e8m0fnu, which appends keep.

    Long chunks of bfloat16 over 8-bit pages make 16-bit pages of them once, in a workspace of
    up to `most_workspace` bytes (2 GiB), and round their weights to bfloat16 as over 16-bit
    pages; where the batch's tables want more, or torch has no such memory left, they
    take longer and the weights are rounded to float16.  With most_workspace=0 it is always so,
    and a result does not depend on the memory that is free.

    Calls run on the current stream, or on `stream` (a torch stream or a
    cudaStream_t), on which their outputs and workspaces are then allocated too.
    The pages' device has to be the current one.  Several threads may call on one
    stream.  The operators are for serving: results carry no gradient, also where
    the arguments require one."""

    def __init__(self, kv_heads: int, head_dim: int, page_tokens: int, n_pages: int,
                 dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None,
                 v: Optional[torch.Tensor] = None, device=None,
                 page_dtype: Optional[torch.dtype] = None,
                 k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None,
                 most_workspace: Optional[int] = None):
        self.handle = None
        if most_workspace is not None and most_workspace < 0:
            raise ValueError("most_workspace is not negative")
        if dtype not in _DTYPES:
            raise ValueError("a paged cache holds float16 or bfloat16")
        held = dtype if page_dtype is None else page_dtype
        if held is not dtype and held is not _CODES:
            raise ValueError("page_dtype is the cache's dtype or float8_e4m3fn")
        shape = (n_pages, page_tokens, kv_heads, head_dim)
        if (k is None) != (v is None):
            raise ValueError("give both k and v, or neither")
        codes = held is _CODES
        if (k_scales is None) != (v_scales is None) or (k_scales is not None) != (
                codes and k is not None):
            raise ValueError("codes that are given come with k_scales and v_scales, and nothing "
                             "else does")
        if k is None:
            device = device or torch.device("cuda", torch.cuda.current_device())
            k = torch.empty(shape, dtype=held, device=device)
            v = torch.empty(shape, dtype=held, device=device)
            if codes:
                k_scales, v_scales = (torch.empty((n_pages, kv_heads), dtype=_SCALES,
                                                  device=device) for _ in range(2))
        for t in (k, v):
            if tuple(t.shape) != shape or t.dtype != held or not t.is_cuda or t.stride(3) != 1:
                raise ValueError("k and v must be device tensors [n_pages, page_tokens, kv_heads, "
                                 "head_dim] of the cache's type, each head contiguous")
        if k.stride() != v.stride() or k.device != v.device:
            raise ValueError("k and v must have the same strides and device")
        for t in (k_scales, v_scales) if codes else ():
            if (tuple(t.shape) != (n_pages, kv_heads) or t.dtype != _SCALES
                    or t.device != k.device or not t.is_contiguous()):
                raise ValueError("k_scales and v_scales must be contiguous float8_e8m0fnu "
                                 "[n_pages, kv_heads] on the pages' device")
        self.kv_heads, self.head_dim, self.page_tokens = kv_heads, head_dim, page_tokens
        self.n_pages, self.dtype, self.page_dtype, self.k, self.v = n_pages, dtype, held, k, v
        self.k_scales, self.v_scales = k_scales, v_scales
        self.most_workspace = most_workspace
        # whether chunks may be long enough to make 16-bit pages of these
        self._widens = codes and dtype is torch.bfloat16
        self.device, self._index = k.device, k.device.index
        self._bounds_shape = (n_pages, kv_heads, 2, head_dim)
        # a dimension of one element has no stride to speak of
        size = 1 if codes else 2
        row = head_dim * size
        st = [s * size if n > 1 else max(s * size, row) for s, n in zip(k.stride(), shape)]
        desc = ibp.ibp_paged_desc(k.data_ptr(), v.data_ptr(), st[0], st[2], st[1], n_pages,
                                  page_tokens, kv_heads, head_dim, _DTYPES[dtype])
        self._lib = ibp._lib_handle()
        with torch.cuda.device(self._index):  # the handle belongs to the pages' device
            self.handle = (ibp.ibp_paged_create_8bit(desc, k_scales.data_ptr(),
                                                     v_scales.data_ptr())
                           if codes else ibp.ibp_paged_create(desc))

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

    def tables(self, n_seqs: int, max_pages: int) -> "PageTables":
        """Page tables of n_seqs sequences of up to max_pages pages each, on the cache's
        device: every sequence is empty, every page free."""
        return PageTables(self, n_seqs, max_pages)

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
        size = ibp.PAGED_WORKSPACE_BYTES
        # The library says whether a batch's chunks make 16-bit pages; sequences of at most 16 rows
        # of queries to a K/V head are no chunks.
        if (self._widens and pages is None
                and batch.desc.max_q_tokens * heads > 16 * self.kv_heads):
            want = ctypes.c_uint64(0)
            self._lib.ibp_paged_workspace(self.handle, batch.address, heads, ctypes.byref(want))
            most = _MOST_WORKSPACE if self.most_workspace is None else self.most_workspace
            if size < want.value <= most:
                size = want.value
        ws = None
        if size != ibp.PAGED_WORKSPACE_BYTES:
            try:
                ws = _large_workspace(self.device, size)
            except torch.OutOfMemoryError:  # (the call does without)
                size = ibp.PAGED_WORKSPACE_BYTES
        if ws is None:
            ws = _workspace(self.device, raw)
        ibp._check(self._lib.ibp_paged_attention(
            self.handle, batch.address, q.data_ptr(), qs, heads, out.data_ptr(),
            total.data_ptr() if lse else None,
            1.0 / math.sqrt(self.head_dim) if scale is None else scale, 1 if causal else 0, window,
            None if pages is None else pages.data_ptr(), n, ws.data_ptr(), size, raw),
            "ibp_paged_attention")
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


class PageTables:
    """The pages that sequences of a cache hold, kept on the device: page_table [n_seqs,
    max_pages], kv_lens [n_seqs], and the free pages free_pages[:n_free], int32.

    Every sequence is empty at first and every page free; the tensors may be filled in
    otherwise before a call.  Calls on the same tables are for one stream.  Several threads may
    call there, one call follows the other; but the tensors, and with them the batch that
    a call returned, are then the last call's."""

    def __init__(self, cache: PagedCache, n_seqs: int, max_pages: int):
        if n_seqs < 1 or max_pages < 1:
            raise ValueError("page tables have sequences and columns")
        self.cache, self.n_seqs, self.max_pages = cache, n_seqs, max_pages
        dev = cache.device
        self.page_table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=dev)
        self.kv_lens = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.free_pages = torch.arange(cache.n_pages, dtype=torch.int32, device=dev).flip(0)
        self._state = torch.tensor([cache.n_pages, 0], dtype=torch.int32, device=dev)
        self.n_free = self._state[:1]
        self.q_starts = torch.zeros(n_seqs + 1, dtype=torch.int32, device=dev)
        self._batches = {}  # of calls with as many tokens: the tensors are always these
        self._desc = ibp.ibp_paged_tables(
            self.page_table.data_ptr(), self.kv_lens.data_ptr(), self.free_pages.data_ptr(),
            self._state.data_ptr(), max_pages, n_seqs, max_pages)
        self._address = ctypes.addressof(self._desc)

    def resize(self, target: torch.Tensor, n_tokens: int = 0,
               max_q_tokens: Optional[int] = None, slots: Optional[torch.Tensor] = None,
               stream=None) -> Optional[Tuple[PagedBatch, torch.Tensor]]:
        """Sequence s gets target[s] tokens (int32 [n_seqs] on the device): pages come from the
        free ones or go back to them.  n_tokens: rows of the new tokens' arrays, at least
        what sequences grow by together; of one at most max_q_tokens (n_tokens: give it, 1 for a
        step of single tokens, or attention takes each for a chunk and is slower).  Returns the
        batch of the new tokens, whose tensors are these tables' (another call changes them), and
        their slots (int64 [n_tokens]: page * page_tokens + place, rows of key_rows() and
        value_rows(); behind the last new token's they stay as they were); nothing when n_tokens
        is 0: such a call only shrinks.

        Where that cannot be done as a whole nothing changes, the batch is empty (no slot is
        written either), and the cache's status says IBP_ERANGE."""
        if stream is not None:
            with torch.cuda.stream(_as_stream(stream)):
                return self.resize(target, n_tokens, max_q_tokens, slots)
        cache, index = self.cache, self.cache._index
        if (target.shape != self.kv_lens.shape or target.dtype != torch.int32
                or target.get_device() != index or not target.is_contiguous()):
            raise ValueError("target must be a contiguous int32 [n_seqs] on the cache's device")
        if n_tokens <= 0:
            if n_tokens or slots is not None:
                raise ValueError("n_tokens is not negative, and a call without new tokens has no "
                                 "slots")
            ibp._check(cache._lib.ibp_paged_resize(
                cache.handle, self._address, target.data_ptr(), None, None, 0,
                _raw_stream(index)), "ibp_paged_resize")
            return None
        if slots is None:
            slots = torch.empty(n_tokens, dtype=torch.int64, device=cache.device)
        elif (slots.shape != (n_tokens,) or slots.dtype != torch.int64
              or slots.get_device() != index or not slots.is_contiguous()):
            raise ValueError("slots must be a contiguous int64 [n_tokens] on the cache's device")
        ibp._check(cache._lib.ibp_paged_resize(
            cache.handle, self._address, target.data_ptr(), self.q_starts.data_ptr(),
            slots.data_ptr(), n_tokens, _raw_stream(index)), "ibp_paged_resize")
        most = n_tokens if max_q_tokens is None else max_q_tokens
        batch = self._batches.get((n_tokens, most))
        if batch is None:
            if len(self._batches) >= 64:  # (prompts of ever other lengths)
                self._batches.clear()
            batch = self._batches[n_tokens, most] = PagedBatch(
                self.page_table, self.kv_lens, self.q_starts, n_tokens, most)
        return batch, slots
