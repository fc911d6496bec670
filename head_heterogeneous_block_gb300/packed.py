"""Dense causal attention of packed prompts over the C ABI's
``sparse_attn_packed_*`` calls."""
from __future__ import annotations

import ctypes
import math

import torch

from . import PackedShape, _check, _lib, sparse_attn_packed_workspace_size
from ._device import DeviceOperator

_forward = _lib.sparse_attn_packed_forward


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

    def _size(self, tokens, batch, keys):
        """Grow the workspace to what calls of these sizes need, and those so
        far; the device is current."""
        tokens, batch = max(tokens, self._tokens), max(batch, self._batch)
        keys = max(keys, self._keys)
        self._need(sparse_attn_packed_workspace_size(PackedShape(
            total_q=tokens, total_k=keys, batch=batch, num_q_heads=self.num_q_heads,
            num_kv_heads=self.num_kv_heads, head_dim=self.head_dim, scale=self.scale)))
        self._tokens, self._batch, self._keys = tokens, batch, keys

    def __call__(self, q, k, v, cu_q, cu_k=None, out=None, lse=None, stream=None):
        """q bf16 [tokens, num_q_heads, d]; k, v bf16 [keys, num_kv_heads, d]
        (any strides that are multiples of 8, d contiguous).  Sequence s has the
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
        heads, kv_heads, d = self.num_q_heads, self.num_kv_heads, self.head_dim
        qp, q0, q1 = self._rows(q, heads, d, "q")
        kp, k0, k1 = self._rows(k, kv_heads, d, "k")
        vp, v0, v1 = self._rows(v, kv_heads, d, "v")
        tokens, keys, ends = q.shape[0], k.shape[0], cu_q.numel()
        if v.shape[0] != keys:
            raise ValueError("k and v must have the same number of tokens")
        if ends < 2:
            raise ValueError("cu_q must be [batch + 1]")
        cq = self._own(cu_q, torch.int32, (ends,), "cu_q")
        ck = cq if cu_k is None else self._own(cu_k, torch.int32, (ends,), "cu_k")
        if out is None:
            out = torch.empty(tokens, heads, d, dtype=torch.bfloat16, device=self.device)
        op, o0, o1 = self._rows(out, heads, d, "out")
        if out.shape[0] != tokens:
            raise ValueError("out must have q's shape")
        lp = self._own(lse, torch.float32, (tokens, heads), "lse")
        if tokens > self._tokens or ends - 1 > self._batch or keys > self._keys:
            self._size(tokens, ends - 1, keys)
        shape = PackedShape(q0, q1, k0, k1, v0, v1, o0, o1, tokens, keys, ends - 1, heads, kv_heads,
                            d, self.scale)
        status = _forward(ctypes.byref(shape), qp, kp, vp, cq, ck, op, lp, self._ws_ptr, self._ws_bytes,
                          self._status, self._handle())
        if status:
            _check(status, "sparse_attn_packed_forward")
        return out
