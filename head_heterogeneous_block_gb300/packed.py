"""Dense causal attention of packed prompts over the C ABI's
``sparse_attn_packed_*`` calls."""
from __future__ import annotations

import math

import torch

from . import PackedShape, SparseAttnError, _check, sparse_attn_packed_workspace_size
from ._device import NEEDS_WORKSPACE, DeviceOperator, calls


class PackedAttention(DeviceOperator):
    """Causal attention of sequences of different lengths, packed one behind
    the other: grouped query heads, every key (the block-sparse ``PrefillLayer``
    takes one sequence and the blocks that its plan selects).

    ``scale`` of the scores: 1 / sqrt(head_dim) by default.  ``tokens``,
    ``batch`` and ``keys`` (default: ``tokens``) size the workspace ahead of the
    first call (before a graph capture, say) for calls of up to so many queries,
    sequences and keys."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, scale=None, tokens=0, batch=1,
                 keys=None, device="cuda"):
        super().__init__(device)
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else float(scale)
        self._tokens = self._batch = self._keys = 0
        with torch.cuda.device(self.device):
            self._size(tokens, batch, tokens if keys is None else keys)
        self._made()

    def _size(self, tokens, batch, keys):
        """Grow the workspace to what calls of these sizes need, and those so
        far; the device is current."""
        tokens, batch = max(tokens, self._tokens), max(batch, self._batch)
        keys = max(keys, self._keys)
        self._need(sparse_attn_packed_workspace_size(PackedShape(
            total_q=tokens, total_k=keys, batch=batch, num_q_heads=self.num_q_heads,
            num_kv_heads=self.num_kv_heads, head_dim=self.head_dim, scale=self.scale)))
        self._tokens, self._batch, self._keys = tokens, batch, keys
        self._sizes = (self._index, self.num_q_heads, self.num_kv_heads, self.head_dim, self.scale,
                       tokens, batch, keys)

    def __call__(self, q, k, v, cu_q, cu_k=None, out=None, lse=None, stream=None):
        """q bf16 [tokens, num_q_heads, d]; k, v bf16 [keys, num_kv_heads, d]
        (strides multiples of 8, at least head_dim and below 2^38, d contiguous,
        16-byte aligned; a head that several share is given once).  Sequence s has the
        rows ``cu_q[s]`` to ``cu_q[s + 1]`` of q and ``cu_k[s]`` to ``cu_k[s +
        1]`` of k and v (int32 [batch + 1]; ``cu_k``: ``cu_q`` by default).  Its
        queries are its last tokens: with n queries and m keys, query i sees the
        first i + m - n + 1 keys; one that sees none gets zeros.  Returns
        ``out`` (bf16, q's shape; without one a new tensor, whose rows behind
        the last sequence are not written).  ``lse``: fp32 [tokens,
        num_q_heads], written when given.  The lengths are read on the device: a
        captured call follows them."""
        if self._elsewhere(stream):
            return self._on(stream, lambda: self(q, k, v, cu_q, cu_k, out, lse))
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=self.device)
        status = calls.packed(*self._sizes, q, k, v, cu_q, cu_k, out, lse, self._ws_ptr,
                              self._ws_bytes, self._status, self._handle())
        if status == NEEDS_WORKSPACE:
            # in powers of two, so that calls that grow step by step grow it a few times (keys
            # from their own number on: many of them need several times the workspace)
            sizes = q.shape[0], cu_q.numel() - 1, k.shape[0]
            try:
                self._size(*(1 << (max(n, least) - 1).bit_length()
                             for n, least in zip(sizes, (8192, 64, 1024))))
            except SparseAttnError:      # beyond what a call may have: as it is
                self._size(*sizes)
            return self(q, k, v, cu_q, cu_k, out, lse)
        if status:
            _check(status, "sparse_attn_packed_forward")
        return out
