"""A scale that has no finite value in base 2, where exponents are made, is refused."""
import ctypes

import pytest

from tests.test_serving_cpu import _packed, _packed_shape, sa  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_out_of_range_in_base_2(sa, scale):  # noqa: F811
    assert _packed(sa, _packed_shape(sa, scale=scale)) == 1


@pytest.mark.parametrize("scale", [2.3e38, 1e-38])
def test_scales_in_range(sa, scale):  # noqa: F811
    # (without a device the workspace's size is not known: that, and not the shape, is refused)
    n = ctypes.c_size_t()
    assert sa._lib.sparse_attn_packed_workspace_size(ctypes.byref(_packed_shape(sa, scale=scale)), ctypes.byref(n)) != 1
