"""The binding's functions for pages, rotary positions and packed attention raise on
a refusal, before anything touches a device."""
import pytest

from tests.test_serving_cpu import P, _desc, _packed_shape, _pool, _rot, sa  # noqa: F401


def test_binding_functions_raise_on_a_refusal(sa):  # noqa: F811
    q, k = (1024, 128), (256, 128)

    def refused(status, call, *args, **kw):
        with pytest.raises(sa.SparseAttnError) as e:
            call(*args, stream=0, **kw)
        assert e.value.status == status and call.__name__ in str(e.value)

    refused(1, sa.sparse_attn_packed_forward, _packed_shape(sa), P, 2 * P, 3 * P, P, P, P, None, P, 1 << 40, P)
    refused(3, sa.sparse_attn_packed_forward, _packed_shape(sa, head_dim=96), P, 2 * P, 3 * P, P, P, 4 * P, None, P,
            1 << 40, P)
    refused(1, sa.sparse_attn_rotary, _rot(sa), 4, 8, 2, P, P, q, 2 * P, k, 3 * P, q, None, None)
    refused(2, sa.sparse_attn_rotary, _rot(sa), -1, 8, 2, P, P, q, 2 * P, k, 3 * P, q, 4 * P, k)
    refused(1, sa.sparse_attn_rotary_store, _rot(sa), 4, 8, P, P, q, 2 * P, k, 5 * P, k, 3 * P, q, None, None, _desc(sa),
            None, P)
    growth = sa.PageGrowth(cu=P, slots=8 * P, lens_out=P, owned_out=P, free_count_out=P, tokens=10)
    refused(1, sa.sparse_attn_paged_grow, _pool(sa), growth, P, 100, P)
    refused(3, sa.sparse_attn_paged_grow, _pool(sa, page=48), growth, P, 1 << 40, P)
    with pytest.raises(sa.SparseAttnError):
        sa.sparse_attn_packed_workspace_size(_packed_shape(sa, batch=0))
    with pytest.raises(sa.SparseAttnError):
        sa.sparse_attn_paged_grow_workspace_size(_pool(sa, page=48))
