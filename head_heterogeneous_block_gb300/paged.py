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


def _need(ok, what):
    if not ok:
        raise ValueError(what)


class PagedCache:
    """Tensors of a paged cache, all on one CUDA device:

    ``k_pages``, ``v_pages``  bf16 [num_pages, page, d]; a page is contiguous,
                  pages may be any multiple of 8 elements apart
    ``table``     int32 [batch, num_kv_heads, max_pages] page numbers
    ``lens``      int32 [batch, num_kv_heads] tokens of each row
    ``weights``   fp32 [batch, num_kv_heads, max_pages * page], or None
    ``positions`` int32 of the same shape, or None

    ``num_q_heads`` only sizes the workspace ahead of the first ``attend``
    (before a graph capture, say).  The calls of one PagedCache share its
    workspace: they must not run at the same time on several streams.
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
            if t.dtype != dtype:
                raise TypeError(f"{name} must be {dtype}")
            _need(t.dim() == nd, f"{name} must have {nd} dimensions")
            _need(t.device == dev, f"{name} must be on {dev}")
        _need(dev.type == "cuda", "the cache's tensors must be on a CUDA device")
        pages, page, d = k_pages.shape
        _need(v_pages.shape == k_pages.shape, "k_pages and v_pages must have the same shape")
        for t in (k_pages, v_pages):
            _need(t.stride(2) == 1 and t.stride(1) == d, "a page must be contiguous")
        b, h, max_pages = table.shape
        _need(tuple(lens.shape) == (b, h), "lens must be [batch, num_kv_heads]")
        for name, t in (("table", table), ("lens", lens), ("weights", weights),
                        ("positions", positions)):
            _need(t is None or t.is_contiguous(), f"{name} must be contiguous")
        self.slots = max_pages * page
        for name, t in (("weights", weights), ("positions", positions)):
            _need(t is None or tuple(t.shape) == (b, h, self.slots),
                  f"{name} must be [batch, num_kv_heads, max_pages * page]")
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
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._status = self.dev_status.data_ptr()
        self._ws = None
        self._ws_bytes = 0
        self._ws_stream = torch.cuda.current_stream(dev).cuda_stream
        self._need_ws = {}
        if num_q_heads is not None:
            self._workspace(("attend", num_q_heads, weights is not None))
        if weights is not None:
            self._workspace(("evict",))

    # -- helpers
    def _workspace(self, key):
        need = self._need_ws.get(key)
        if need is None:
            with torch.cuda.device(self.device):
                need = (sparse_attn_paged_evict_workspace_size(self.desc) if key[0] == "evict" else
                        sparse_attn_paged_attend_workspace_size(self.desc, key[1], key[2]))
            self._need_ws[key] = need
        if need > self._ws_bytes:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            self._ws_bytes = need
            self._ws_stream = torch.cuda.current_stream(self.device).cuda_stream
        return self._ws.data_ptr()

    def _call(self, fn, stream, *args):
        """fn(*args, stream) with the cache's device current."""
        dev = self.device
        if torch.cuda.current_device() != dev.index:
            with torch.cuda.device(dev):
                return self._call(fn, stream, *args)
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(dev.index)
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if handle != self._ws_stream:
            # the cache's own tensors outlive the work of streams they were
            # not allocated on
            other = torch.cuda.ExternalStream(handle, device=dev)
            self.dev_status.record_stream(other)
            if self._ws is not None:
                self._ws.record_stream(other)
        status = fn(*args, handle)
        if status:
            _check(status, fn.__name__)

    def _row_array(self, t, dtype, shape, name):
        if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}")
        return t.data_ptr()

    # -- the three operators
    def append(self, k, v, counts=None, start=None, lens_out=None, stream=None):
        """Append ``counts[b]`` (default: all) of the tokens of ``k``, ``v``
        (bf16 [batch, num_kv_heads, tokens, d], any strides that are multiples
        of 8, d contiguous) to every row of sequence b, at positions
        ``start[b]``, ``start[b]`` + 1, ... (default: their slots).  The new
        lengths go to ``lens_out`` (default: ``lens``)."""
        b, h, d = self.batch, self.num_kv_heads, self.head_dim
        for name, t in (("k", k), ("v", v)):
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be bfloat16")
            _need(t.dim() == 4 and t.shape[0] == b and t.shape[1] == h and t.shape[3] == d and
                  t.shape[2] >= 1 and t.stride(3) == 1,
                  f"{name} must be [batch, num_kv_heads, tokens, d] with d contiguous")
            _need(t.device == self.device, f"{name} must be on {self.device}")
        tokens = k.shape[2]
        _need(v.shape[2] == tokens, "k and v must have the same shape")
        strides = [_I64x3(*(st if n > 1 else 0 for st, n in zip(t.stride(), t.shape[:3])))
                   for t in (k, v)]
        self._call(_lib.sparse_attn_paged_append, stream, self._ref, k.data_ptr(), v.data_ptr(),
                   strides[0], strides[1], tokens,
                   None if counts is None else self._row_array(counts, torch.int32, (b,), "counts"),
                   None if start is None else self._row_array(start, torch.int32, (b,), "start"),
                   self.desc.lens if lens_out is None else
                   self._row_array(lens_out, torch.int32, (b, h), "lens_out"),
                   self._status)

    def attend(self, q, out=None, lse=None, weights_out=None, accumulate=None, stream=None):
        """Attention of one new token per sequence: q bf16 [batch, num_q_heads,
        d] (strides multiples of 8, d contiguous) over every row's tokens.
        Returns ``out`` (bf16 or fp32 [batch, num_q_heads, d]; a new bf16
        tensor when None).  ``lse``: fp32 [batch, num_q_heads], written when
        given.  ``accumulate`` (default: when the cache has weights) adds each
        token's probability, summed over the row's heads, to its weight, into
        ``weights_out`` (default: ``weights``)."""
        b, d = self.batch, self.head_dim
        if q.dtype != torch.bfloat16:
            raise TypeError("q must be bfloat16")
        _need(q.dim() == 3 and q.shape[0] == b and q.shape[2] == d and q.stride(2) == 1,
              "q must be [batch, num_q_heads, d] with d contiguous")
        _need(q.device == self.device, f"q must be on {self.device}")
        hq = q.shape[1]
        if out is None:
            out = torch.empty(b, hq, d, dtype=torch.bfloat16, device=self.device)
            if stream is not None and not isinstance(stream, int):
                out.record_stream(stream)
        if out.dtype == torch.bfloat16:
            o_dtype = SA_DTYPE_BF16
        elif out.dtype == torch.float32:
            o_dtype = SA_DTYPE_F32
        else:
            raise TypeError("out must be bfloat16 or float32")
        o = self._row_array(out, out.dtype, (b, hq, d), "out")
        if lse is not None:
            lse = self._row_array(lse, torch.float32, (b, hq), "lse")
        if accumulate is None:
            accumulate = self.weights is not None
        w = None
        if accumulate:
            _need(self.weights is not None, "the cache has no weights to accumulate into")
            w = (self.desc.weights if weights_out is None else
                 self._row_array(weights_out, torch.float32, tuple(self.weights.shape),
                                 "weights_out"))
        else:
            _need(weights_out is None, "weights_out needs accumulate")
        ws = self._workspace(("attend", hq, bool(accumulate)))
        self._call(_lib.sparse_attn_paged_attend, stream, self._ref, q.data_ptr(), q.stride(0),
                   q.stride(1), hq, o, o_dtype, lse, w, ws, self._ws_bytes, self._status)
        return out

    def evict(self, keep, sinks=0, recent=0, lens_out=None, weights_out=None, positions_out=None,
              stream=None):
        """Cut every row of KV head g to at most ``keep[g]`` tokens (ints): the
        first ``sinks`` positions, the last ``recent`` ones, then the largest
        weights.  The new state goes to ``lens_out``, ``weights_out`` and
        ``positions_out`` (default: the cache's own tensors)."""
        _need(self.weights is not None, "eviction needs the cache's weights")
        _need(len(keep) == self.num_kv_heads, "keep must hold one budget per KV head")
        shape = tuple(self.weights.shape)
        if positions_out is not None:
            _need(self.positions is not None, "positions_out needs the cache's positions")
        ws = self._workspace(("evict",))
        self._call(_lib.sparse_attn_paged_evict, stream, self._ref,
                   (ctypes.c_int32 * len(keep))(*keep), sinks, recent,
                   self.desc.lens if lens_out is None else
                   self._row_array(lens_out, torch.int32, (self.batch, self.num_kv_heads),
                                   "lens_out"),
                   self.desc.weights if weights_out is None else
                   self._row_array(weights_out, torch.float32, shape, "weights_out"),
                   self.desc.positions if positions_out is None else
                   self._row_array(positions_out, torch.int32, shape, "positions_out"),
                   ws, self._ws_bytes, self._status)
