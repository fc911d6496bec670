"""A paged key-value cache over the C ABI's ``sparse_attn_paged_*`` calls.

``PagedCache`` binds tensors that the caller owns: the page pools, the page
table and the lengths of every (sequence, KV head) row, and, for eviction, the
slots' accumulated weights and positions.  Every step of the computation runs
in libsparse_attn's kernels; the class checks shapes and keeps the workspace.
``layer.PagedDecodeLayer`` also hands out the pages.
"""
from __future__ import annotations

import ctypes

import torch

from . import (SA_DTYPE_BF16, SA_DTYPE_F32, PagedCacheDesc, _check, _lib,
               sparse_attn_paged_attend_workspace_size, sparse_attn_paged_evict_workspace_size)

_I64x3 = ctypes.c_int64 * 3
_INT32_MAX = 2**31 - 1
# what eviction serves (attention goes further)
MAX_EVICT_SLOTS, MAX_EVICT_KV_HEADS = 262144, 256
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_append, _attend, _evict = (_lib.sparse_attn_paged_append, _lib.sparse_attn_paged_attend,
                            _lib.sparse_attn_paged_evict)


class PagedCache:
    """Tensors of a paged cache, all on one CUDA device:

    ``k_pages``, ``v_pages``  bf16 [num_pages, page, d]; a page is contiguous,
                  pages may be any multiple of 8 elements apart
    ``table``     int32 [batch, num_kv_heads, max_pages] page numbers
    ``lens``      int32 [batch, num_kv_heads] tokens of each row
    ``weights``   fp32 [batch, num_kv_heads, max_pages * page], or None
    ``positions`` int32 of the same shape, or None

    ``num_q_heads`` only sizes the workspace ahead of the first ``attend``
    (before a graph capture, say).  Rows of more than 262144 slots, or more
    than 256 KV heads, can have weights but not be evicted from.  The calls of one PagedCache share its
    workspace: they must not run at the same time on several streams, nor may
    the replays of graphs that hold them.  A graph that captured a call needs
    its PagedCache, and its tensors, to live.
    ``dev_status`` collects the device's error bits (``SA_DEV_*``)."""

    def __init__(self, k_pages, v_pages, table, lens, weights=None, positions=None,
                 num_q_heads=None):
        dev = k_pages.device
        self.device = dev
        for name, t, dtype, nd in (("k_pages", k_pages, torch.bfloat16, 3),
                                   ("v_pages", v_pages, torch.bfloat16, 3),
                                   ("table", table, torch.int32, 3),
                                   ("lens", lens, torch.int32, 2),
                                   ("weights", weights, torch.float32, 3),
                                   ("positions", positions, torch.int32, 3)):
            if t is None:
                continue
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}")
            if t.dim() != nd:
                raise ValueError(f"{name} must have {nd} dimensions")
            if t.device != dev:
                raise ValueError(f"{name} must be on {dev}")
            if t is not k_pages and t is not v_pages and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if dev.type != "cuda":
            raise ValueError("the cache's tensors must be on a CUDA device")
        pages, page, d = k_pages.shape
        if v_pages.shape != k_pages.shape:
            raise ValueError("k_pages and v_pages must have the same shape")
        for t in (k_pages, v_pages):
            if t.stride(2) != 1 or t.stride(1) != d:
                raise ValueError("a page must be contiguous")
        b, h, max_pages = table.shape
        if tuple(lens.shape) != (b, h):
            raise ValueError("lens must be [batch, num_kv_heads]")
        self.slots = max_pages * page
        for name, t in (("weights", weights), ("positions", positions)):
            if t is not None and tuple(t.shape) != (b, h, self.slots):
                raise ValueError(f"{name} must be [batch, num_kv_heads, max_pages * page]")
        self.k_pages, self.v_pages, self.table, self.lens = k_pages, v_pages, table, lens
        self.weights, self.positions = weights, positions
        self.batch, self.num_kv_heads, self.head_dim, self.page = b, h, d, page
        one = page * d                 # a single page's stride is not used
        self.desc = PagedCacheDesc(
            k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(),
            weights.data_ptr() if weights is not None else None,
            positions.data_ptr() if positions is not None else None, pages,
            k_pages.stride(0) if pages > 1 else one, v_pages.stride(0) if pages > 1 else one,
            page, max_pages, b, h, d)
        self._ref = ctypes.byref(self.desc)
        self._index = k_pages.get_device()
        self._shape_b, self._shape_lens = torch.Size((b,)), torch.Size((b, h))
        self._keep = ctypes.c_int32 * h
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._status = self.dev_status.data_ptr()
        self._ws, self._ws_ptr, self._ws_bytes = None, None, 0
        self._outgrown = []
        # the streams that the status word and the workspace were allocated on,
        # and the one that both were (None: they differ)
        self._status_stream = self._ws_stream = self._home = _raw_stream(self._index)
        self._sized = set()
        if num_q_heads is not None:
            self._size(num_q_heads, weights is not None)
        if weights is not None and self.slots <= MAX_EVICT_SLOTS and h <= MAX_EVICT_KV_HEADS:
            self._size()
        # what was queued here, and by the last owners of its memory before, is done: a
        # call may go to any stream
        with torch.cuda.device(self.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    # -- helpers (a step's calls are short: checks are written out where a
    # call per check, or a message built for nothing, would cost more)
    def _size(self, num_q_heads=None, accumulate=False):
        """Grow the workspace to what ``attend`` with these arguments (None:
        ``evict``) needs."""
        if _current_device() != self._index:
            with torch.cuda.device(self.device):
                return self._size(num_q_heads, accumulate)
        need = (sparse_attn_paged_evict_workspace_size(self.desc) if num_q_heads is None else
                sparse_attn_paged_attend_workspace_size(self.desc, num_q_heads, accumulate))
        if need > self._ws_bytes:
            if self._ws is not None:        # graphs captured with it still use it
                self._outgrown.append(self._ws)
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            self._ws_ptr, self._ws_bytes = self._ws.data_ptr(), need
            self._ws_stream = _raw_stream(self._index)
            self._home = self._ws_stream if self._ws_stream == self._status_stream else None
        self._sized.add((num_q_heads, accumulate))

    def _stream(self, handle):
        # (an external stream of handle 0 would be a new stream)
        return (torch.cuda.ExternalStream(handle, device=self.device) if handle else
                torch.cuda.default_stream(self.device))

    def _given(self, stream):
        """Handle of a ``stream`` argument: a handle, or a stream of the
        cache's device."""
        if isinstance(stream, int):
            return stream
        if stream.device_index != self._index:
            raise ValueError(f"stream must be on {self.device}")
        return stream.cuda_stream

    def _handle(self, stream):
        """The stream's handle; the cache's device is current."""
        handle = _raw_stream(self._index) if stream is None else self._given(stream)
        if handle != self._home:
            # the cache's own tensors outlive the work of streams they were
            # not allocated on
            if handle != self._status_stream:
                self.dev_status.record_stream(self._stream(handle))
            if handle != self._ws_stream and self._ws is not None:
                self._ws.record_stream(self._stream(handle))
        return handle

    def _own(self, t, dtype, shape, name):
        """Address of a contiguous tensor of the cache's device."""
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
        if t.get_device() != self._index:
            raise ValueError(f"{name} must be on {self.device}")
        return t.data_ptr()

    # -- the three operators
    def append(self, k, v, counts=None, start=None, lens_out=None, stream=None):
        """Append ``counts[b]`` (default: all) of the tokens of ``k``, ``v``
        (bf16 [batch, num_kv_heads, tokens, d], any strides that are multiples
        of 8, d contiguous) to every row of sequence b, at positions
        ``start[b]``, ``start[b]`` + 1, ... (default: their slots).  The new
        lengths go to ``lens_out`` (default: ``lens``), which may share memory
        with ``start`` but not with another row's ``counts``."""
        if _current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.append(k, v, counts, start, lens_out, stream)
        b, h, tokens, d = k.shape if k.dim() == 4 else (0, 0, 0, 0)
        if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16:
            raise TypeError("k and v must be bfloat16")
        if b != self.batch or h != self.num_kv_heads or d != self.head_dim or tokens < 1:
            raise ValueError("k must be [batch, num_kv_heads, tokens, d]")
        if v.shape != k.shape:
            raise ValueError("k and v must have the same shape")
        k0, k1, k2, k3 = k.stride()
        v0, v1, v2, v3 = v.stride()
        if k3 != 1 or v3 != 1:
            raise ValueError("the last dimension of k and v must be contiguous")
        if k.get_device() != self._index or v.get_device() != self._index:
            raise ValueError(f"k and v must be on {self.device}")
        if b == 1:                          # the stride of an extent of one is not used
            k0 = v0 = 0
        if h == 1:
            k1 = v1 = 0
        if tokens == 1:
            k2 = v2 = 0
        if counts is not None:
            counts = self._own(counts, torch.int32, self._shape_b, "counts")
        if start is not None:
            start = self._own(start, torch.int32, self._shape_b, "start")
        lens = (self.desc.lens if lens_out is None else
                self._own(lens_out, torch.int32, self._shape_lens, "lens_out"))
        status = _append(self._ref, k.data_ptr(), v.data_ptr(), _I64x3(k0, k1, k2),
                         _I64x3(v0, v1, v2), tokens, counts, start, lens, self._status,
                         self._handle(stream))
        if status:
            _check(status, "sparse_attn_paged_append")

    def attend(self, q, out=None, lse=None, weights_out=None, accumulate=None, stream=None):
        """Attention of one new token per sequence: q bf16 [batch, num_q_heads,
        d] (strides multiples of 8, d contiguous) over every row's tokens.
        Returns ``out`` (bf16 or fp32 [batch, num_q_heads, d]; a new bf16
        tensor when None).  ``lse``: fp32 [batch, num_q_heads], written when
        given.  ``accumulate`` (default: when the cache has weights) adds each
        token's probability, summed over the row's heads, to its weight, into
        ``weights_out`` (default: ``weights``)."""
        if _current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.attend(q, out, lse, weights_out, accumulate, stream)
        if stream is not None and self._given(stream) != _raw_stream(self._index):
            # what is allocated here (the output, a larger workspace) comes from
            # the launching stream's memory: the current stream may still be at
            # work in what it freed
            caller, made = torch.cuda.current_stream(), out is None
            with torch.cuda.stream(self._stream(stream) if isinstance(stream, int) else stream):
                out = self.attend(q, out, lse, weights_out, accumulate)
            if made:
                out.record_stream(caller)
            return out
        if q.dtype is not torch.bfloat16:
            raise TypeError("q must be bfloat16")
        b, hq, d = q.shape if q.dim() == 3 else (0, 0, 0)
        if b != self.batch or d != self.head_dim:
            raise ValueError("q must be [batch, num_q_heads, d]")
        q0, q1, q2 = q.stride()
        if q2 != 1:
            raise ValueError("the last dimension of q must be contiguous")
        if q.get_device() != self._index:
            raise ValueError(f"q must be on {self.device}")
        if out is None:
            out = torch.empty(b, hq, d, dtype=torch.bfloat16, device=self.device)
        if out.dtype is torch.bfloat16:
            o_dtype = SA_DTYPE_BF16
        elif out.dtype is torch.float32:
            o_dtype = SA_DTYPE_F32
        else:
            raise TypeError("out must be bfloat16 or float32")
        o = self._own(out, out.dtype, q.shape, "out")
        if lse is not None:
            lse = self._own(lse, torch.float32, (b, hq), "lse")
        if accumulate is None:
            accumulate = self.weights is not None
        w = None
        if accumulate:
            if self.weights is None:
                raise ValueError("the cache has no weights to accumulate into")
            w = (self.desc.weights if weights_out is None else
                 self._own(weights_out, torch.float32, self.weights.shape, "weights_out"))
        elif weights_out is not None:
            raise ValueError("weights_out needs accumulate")
        if (hq, w is not None) not in self._sized:
            self._size(hq, w is not None)
        status = _attend(self._ref, q.data_ptr(), q0, q1, hq, o, o_dtype, lse, w, self._ws_ptr,
                         self._ws_bytes, self._status, self._handle(None))
        if status:
            _check(status, "sparse_attn_paged_attend")
        return out

    def evict(self, keep, sinks=0, recent=0, lens_out=None, weights_out=None, positions_out=None,
              stream=None):
        """Cut every row of KV head g to at most ``keep[g]`` tokens (ints): the
        first ``sinks`` positions, the last ``recent`` ones, then the largest
        weights.  The new state goes to ``lens_out``, ``weights_out`` and
        ``positions_out`` (default: the cache's own tensors)."""
        if _current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.evict(keep, sinks, recent, lens_out, weights_out, positions_out,
                                  stream)
        if self.weights is None:
            raise ValueError("eviction needs the cache's weights")
        keep = [int(k) for k in keep]
        if len(keep) != self.num_kv_heads or min(keep) < 0 or max(keep) > _INT32_MAX:
            raise ValueError("keep must hold one 32-bit budget per KV head")
        if not (0 <= sinks <= _INT32_MAX and 0 <= recent <= _INT32_MAX):
            raise ValueError("sinks and recent must be 32-bit and not negative")
        if positions_out is not None and self.positions is None:
            raise ValueError("positions_out needs the cache's positions")
        shape = self.weights.shape
        lens = (self.desc.lens if lens_out is None else
                self._own(lens_out, torch.int32, self._shape_lens, "lens_out"))
        w = (self.desc.weights if weights_out is None else
             self._own(weights_out, torch.float32, shape, "weights_out"))
        pos = (self.desc.positions if positions_out is None else
               self._own(positions_out, torch.int32, shape, "positions_out"))
        status = _evict(self._ref, self._keep(*keep), sinks, recent, lens, w, pos,
                        self._ws_ptr, self._ws_bytes, self._status, self._handle(stream))
        if status:
            _check(status, "sparse_attn_paged_evict")


class PageBook:
    """Which pages of a pool belong to which (sequence, KV head) row, on the
    host.  Pages come back when rows shrink, and those that came back last are
    handed out first; nothing here touches the device."""

    def __init__(self, num_pages, page, batch, num_kv_heads, max_pages):
        self.page, self.max_pages = page, max_pages
        self.free = list(range(num_pages - 1, -1, -1))
        self.rows = [[[] for _ in range(num_kv_heads)] for _ in range(batch)]
        self.lens = [[0] * num_kv_heads for _ in range(batch)]

    def _pages(self, tokens):
        return -(-tokens // self.page)

    def missing(self, growth):
        """Pages that rows need to grow by ``growth[b]`` tokens each."""
        return sum(max(0, self._pages(n + growth[b]) - len(row))
                   for b, rows in enumerate(self.rows)
                   for row, n in zip(rows, self.lens[b]))

    def grow(self, growth):
        """Grow every row of sequence b by ``growth[b]`` tokens; returns the new
        table entries as (sequence, KV head, entry, page) tuples.  Nothing
        changes when the pages or the table do not suffice."""
        for b, more in enumerate(growth):
            if more < 0 or (more and max(self.lens[b]) + more > self.max_pages * self.page):
                raise ValueError(f"sequence {b} cannot grow by {more} tokens")
        if self.missing(growth) > len(self.free):
            raise MemoryError(f"the pool has {len(self.free)} free pages, "
                              f"{self.missing(growth)} are needed")
        new = []
        for b, more in enumerate(growth):
            if not more:
                continue
            for g, row in enumerate(self.rows[b]):
                self.lens[b][g] += more
                while len(row) < self._pages(self.lens[b][g]):
                    new.append((b, g, len(row), self.free[-1]))
                    row.append(self.free.pop())
        return new

    def shrink(self, b, lens):
        """Cut sequence b's rows to at most ``lens[g]`` tokens; their spare
        pages are free again."""
        for g, row in enumerate(self.rows[b]):
            self.lens[b][g] = min(self.lens[b][g], lens[g])
            while len(row) > self._pages(self.lens[b][g]):
                self.free.append(row.pop())
