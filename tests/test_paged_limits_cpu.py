"""Argument checks of the paged cache that answer before anything touches a
device: aliases, limits of the eviction, settings of the decode layer."""
import ctypes

import pytest

from tests.test_paged_cpu import P, _append, desc, sa  # noqa: F401  (sa: the fixture)


def test_append_refuses_lengths_over_the_counts(sa):  # noqa: F811
    # 2 sequences of 2 heads: 16 bytes of lengths, 8 of counts
    for at in (P, P + 4, P + 12, P - 4):
        assert _append(sa, desc(sa), counts=at, lens_out=P, start=None) == 1
    assert _append(sa, desc(sa, num_kv_heads=1), counts=P + 4, lens_out=P, start=None) == 1
