"""The pages of a paged cache, accounted for on the device, over the C ABI's
``sparse_attn_paged_grow``."""
from __future__ import annotations

import ctypes

import torch

from . import PagePoolDesc, _check, sparse_attn_paged_grow_workspace_size
from ._device import DeviceOperator, calls


class PagePool(DeviceOperator):
    """Which pages belong to which (sequence, KV head) row, on the device: rows
    grow, shrink and end without the host, so a serving step can be captured
    into a graph (``PagedDecodeLayer`` keeps the same account on the host).

    ``table``       int32 [batch, num_kv_heads, max_pages], as ``PagedCache``'s
    ``lens``        int32 [batch, num_kv_heads], the cache's
    ``page``        tokens of a page
    ``free_pages``  int32 [num_pages]; the first ``free_count`` (int32 [1]) are
                    free.  ``num_pages`` makes them: all pages free, all rows
                    empty
    ``owned``       int32 of ``lens``' shape: table entries that are a row's own
    ``weights``, ``positions``  the cache's, or None: set for new tokens

    ``PagePool.of(cache)`` is the pool of a ``PagedCache`` whose pages are all
    free."""

    def __init__(self, table, lens, page, num_pages=None, free_pages=None, free_count=None,
                 owned=None, weights=None, positions=None):
        super().__init__(table.device)
        if table.dim() != 3:
            raise ValueError("table must be [batch, num_kv_heads, max_pages]")
        b, h, max_pages = table.shape
        given = [t is not None for t in (free_pages, free_count, owned)]
        if any(given) != all(given) or all(given) == (num_pages is not None):
            raise ValueError("give num_pages, or free_pages, free_count and owned")
        if num_pages is not None:
            if not 1 <= num_pages < 2**30:
                raise ValueError("num_pages must be positive and below 2^30")
            free_pages = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=self.device)
            free_count = torch.full((1,), num_pages, dtype=torch.int32, device=self.device)
            owned = torch.zeros(b, h, dtype=torch.int32, device=self.device)
        i32 = torch.int32
        slots = (b, h, max_pages * page)
        self.table, self.lens, self.page = table, lens, page
        self.free_pages, self.free_count, self.owned = free_pages, free_count, owned
        self.weights, self.positions = weights, positions
        self.batch, self.num_kv_heads, self.num_pages = b, h, free_pages.numel()
        self._desc = PagePoolDesc(
            self._own(table, i32, table.shape, "table"), self._own(lens, i32, (b, h), "lens"),
            self._own(owned, i32, (b, h), "owned"),
            self._own(free_pages, i32, (self.num_pages,), "free_pages"),
            self._own(free_count, i32, (1,), "free_count"),
            self._own(weights, torch.float32, slots, "weights"),
            self._own(positions, i32, slots, "positions"), self.num_pages, page, max_pages, b, h)
        self._desc_ptr = ctypes.addressof(self._desc)
        self._own_tensors = () if num_pages is None else (free_pages, free_count, owned)
        with torch.cuda.device(self.device):
            self._need(sparse_attn_paged_grow_workspace_size(self._desc))
        self._made()

    @classmethod
    def of(cls, cache):
        """The pool of a ``PagedCache`` whose rows are all empty (its lengths are
        set to 0) and whose pages are all free."""
        cache.lens.zero_()
        return cls(cache.table, cache.lens, cache.page, num_pages=cache.k_pages.shape[0],
                   weights=cache.weights, positions=cache.positions)

    def grow(self, slots, cu=None, counts=None, ended=None, start=None, positions=None,
             granted=None, lens_out=None, owned_out=None, free_count_out=None, start_out=None,
             stream=None):
        """Pages and slots for new tokens; rows give back pages that they do not
        need.  Sequence b has the tokens ``cu[b]`` to ``cu[b + 1]`` of a packed
        tensor (int32 [batch + 1]), or without ``cu`` an equal span of a padded
        one, and uses the first ``counts[b]`` of them (int32 [batch]; default:
        all).  Sequences where ``ended`` (bool [batch]) is true are emptied
        first.  ``start``: int32 [batch], the positions of the first new tokens
        (0 where ended; default: the sequence's longest row).

        ``slots`` (int64 [num_kv_heads, tokens]) receives each token's slot of
        the pools for ``Rotary.store``, -1 for tokens that get none;
        ``positions`` (int32 [tokens]) the tokens' positions, ``granted`` (int32
        [batch]) how many tokens of each sequence got slots: all, or none where
        the pool has too few pages for it or for one before it
        (``SA_DEV_NO_PAGES``).  The new state goes to ``lens_out``,
        ``owned_out``, ``free_count_out`` and ``start_out`` (default: the pool's
        own tensors, and ``start``)."""
        if self._elsewhere(stream):
            return self._on(stream, lambda: self.grow(
                slots, cu, counts, ended, start, positions, granted, lens_out, owned_out,
                free_count_out, start_out))
        handle = self._handle()
        if handle != self._status_stream:
            for t in self._own_tensors:
                t.record_stream(self._stream(handle))
        status = calls.grow(self._desc_ptr, self._index, slots, cu, counts, ended, start,
                            positions, granted, lens_out, owned_out, free_count_out, start_out,
                            self._ws_ptr, self._ws_bytes, self._status, handle)
        if status:
            _check(status, "sparse_attn_paged_grow")
