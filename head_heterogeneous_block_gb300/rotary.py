"""Rotary positions over the C ABI's ``sparse_attn_rotary*`` calls: the
frequencies and their scalings, and the operator class."""
from __future__ import annotations

import ctypes
import decimal
import math
import operator
from decimal import Decimal

import torch

from . import RotaryDesc, _check
from ._device import DeviceOperator, calls


# 64-bit fractions of a turn need more digits than a double has
_DIGITS = decimal.Context(prec=80)
_TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def rotary_frequencies(rot_dim, base=10000.0, scaling=None):
    """Radians a position of each of the ``rot_dim / 2`` pairs (floats), and the
    factor on the rotated values.  ``scaling`` stretches them for contexts
    longer than the model was trained on: None, or a dict with ``type``

    ``linear``      every frequency divided by ``factor`` (positions interpolated)
    ``ntk``         the base raised to base * factor^(rot_dim / (rot_dim - 2)):
                    the highest frequency stays, the lowest is divided by factor
    ``wavelength``  with the turns that a pair makes over ``original`` positions:
                    below ``low`` divided by factor, above ``high`` kept, between
                    them blended in proportion to the turns
    ``yarn``        kept for pairs of more than ``beta_fast`` (32) turns over
                    ``original`` positions, divided by factor below
                    ``beta_slow`` (1), blended in proportion to the pair's number
                    between them; values times ``attention_factor`` (0.1
                    ln(factor) + 1, and 1 for factors up to 1)
    """
    freq, multiplier = _frequencies(rot_dim, base, scaling)
    return [float(f) for f in freq], multiplier


def _frequencies(rot_dim, base, scaling):
    """As ``rotary_frequencies``, to 80 digits."""
    with decimal.localcontext(_DIGITS):
        return _scaled(rot_dim, base, scaling)


def _turns(freq):
    """Fractions of a turn a position, in 2^-64ths, of what ``_frequencies`` gives."""
    with decimal.localcontext(_DIGITS):
        return [int((f / _TWO_PI * 2**64).to_integral_value()) % 2**64 for f in freq]


def _scaled(rot_dim, base, scaling):
    rot_dim = operator.index(rot_dim)
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    base = float(base)
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError("base must be finite and above 1")
    scaling = dict(scaling) if scaling else {"type": "none"}
    kind = scaling.pop("type", None)

    def get(name, default=None):
        value = scaling.pop(name, default)
        if value is None:
            raise ValueError(f"scaling {kind!r} needs {name!r}")
        if not (float(value) > 0 and math.isfinite(float(value))):
            raise ValueError(f"scaling {name!r} must be positive and finite")
        return float(value)

    multiplier = 1.0
    pairs = range(rot_dim // 2)
    exact = Decimal(base)
    if kind == "ntk":
        factor = get("factor")
        if rot_dim > 2:
            exact *= Decimal(factor) ** (Decimal(rot_dim) / (rot_dim - 2))
    # (one root and its powers: a root each would take milliseconds)
    step, freq = exact ** (Decimal(-2) / rot_dim), [Decimal(1)]
    while len(freq) < len(pairs):
        freq.append(freq[-1] * step)
    if kind == "linear":
        factor = Decimal(get("factor"))
        freq = [f / factor for f in freq]
    elif kind == "wavelength":
        factor, low, high, original = (Decimal(get(x)) for x in ("factor", "low", "high", "original"))
        if not low < high:
            raise ValueError("scaling 'low' must be below 'high'")
        keep = [min(Decimal(1), max(Decimal(0), (f * original / _TWO_PI - low) / (high - low)))
                for f in freq]
        freq = [f * x + f / factor * (1 - x) for f, x in zip(freq, keep)]
    elif kind == "yarn":
        factor, original = get("factor"), get("original")
        fast, slow = get("beta_fast", 32.0), get("beta_slow", 1.0)
        multiplier = get("attention_factor", 0.1 * math.log(max(factor, 1.0)) + 1.0)
        if fast < slow:
            raise ValueError("scaling 'beta_fast' must not be below 'beta_slow'")

        def pair(turns):
            return rot_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot_dim - 1)
        slowed = [min(Decimal(1), max(Decimal(0), Decimal(i - lo) / max(hi - lo, Decimal("0.001"))))
                  for i in pairs]
        freq = [f * (1 - x) + f / Decimal(factor) * x for f, x in zip(freq, slowed)]
    elif kind not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {kind!r}")
    if scaling:
        raise ValueError(f"scaling {kind!r} does not take {sorted(scaling)}")
    return freq, multiplier


class Rotary(DeviceOperator):
    """Rotary positions of queries and keys: the first ``rot_dim`` of
    ``head_dim`` elements (default: all), in pairs (i, i + rot_dim/2) or, with
    ``interleaved``, (2i, 2i + 1).  ``base`` and ``scaling`` as
    ``rotary_frequencies`` takes them."""

    def __init__(self, head_dim, rot_dim=None, base=10000.0, interleaved=False, scaling=None,
                 device="cuda"):
        rot_dim = head_dim if rot_dim is None else rot_dim
        if head_dim not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if rot_dim % 16 or not 16 <= rot_dim <= head_dim:
            raise ValueError("rot_dim must be a multiple of 16 up to head_dim")
        freq, self.factor = _frequencies(rot_dim, base, scaling)
        self.frequencies = [float(f) for f in freq]
        super().__init__(device)
        self.head_dim, self.rot_dim, self.interleaved = head_dim, rot_dim, bool(interleaved)
        # (as the signed 64-bit numbers of torch)
        self.turns = torch.tensor([t - 2**64 if t >= 2**63 else t for t in _turns(freq)],
                                  dtype=torch.int64, device=self.device)
        self._desc = RotaryDesc(self.turns.data_ptr(), self.factor, head_dim, rot_dim,
                                int(self.interleaved))
        self._desc_ptr = ctypes.addressof(self._desc)
        self._made()

    def _follow(self):
        handle = self._handle()
        if handle != self._status_stream:
            self.turns.record_stream(self._stream(handle))
        return handle

    def _like(self, t):
        return torch.empty(t.shape, dtype=torch.bfloat16, device=self.device)

    def __call__(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """q bf16 [tokens, num_q_heads, d], k bf16 [tokens, num_kv_heads, d]
        (strides multiples of 8 below 2^38, 0 among them, d contiguous, 16-byte
        aligned) and positions int32 [tokens].  Returns (``q_out``, ``k_out``:
        their strides at least head_dim): new tensors without them; each may be
        its input, which then changes in place."""
        if self._elsewhere(stream):
            return self._on(stream, lambda: self(q, k, positions, q_out, k_out))
        q_out = self._like(q) if q_out is None else q_out
        k_out = self._like(k) if k_out is None else k_out
        status = calls.rotary(self._desc_ptr, self._index, self.head_dim, q, k, positions, q_out,
                              k_out, self._follow())
        if status:
            _check(status, "sparse_attn_rotary")
        return q_out, k_out

    def store(self, q, k, v, positions, cache, slots, q_out=None, k_out=None, stream=None):
        """As a call, and in the same pass each token's rotated key and its value
        (v bf16 [tokens, num_kv_heads, d]) go to ``slots`` of ``cache`` (a
        ``PagedCache``): int64 [num_kv_heads, tokens], as ``PagePool.grow`` makes
        them; nothing is stored where a slot is -1.  Without ``k_out`` the cache
        has the only copy of the rotated keys.  Returns (``q_out``, ``k_out``).
        A slot outside the pools stores nothing and sets ``SA_DEV_BAD_INDEX`` in
        ``dev_status``."""
        if self._elsewhere(stream):
            return self._on(stream, lambda: self.store(q, k, v, positions, cache, slots, q_out,
                                                       k_out))
        if cache.head_dim != self.head_dim:
            raise ValueError(f"the cache's head_dim must be {self.head_dim}")
        if cache.device != self.device:
            raise ValueError(f"the cache must be on {self.device}")
        q_out = self._like(q) if q_out is None else q_out
        status = calls.rotary_store(self._desc_ptr, self._index, self.head_dim,
                                    cache.num_kv_heads, q, k, v, positions,
                                    ctypes.addressof(cache.desc), slots, q_out, k_out,
                                    self._status, self._follow())
        if status:
            _check(status, "sparse_attn_rotary_store")
        return q_out, k_out
