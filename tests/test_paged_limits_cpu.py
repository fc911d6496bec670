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


@pytest.mark.parametrize("change,status", [
    (dict(), 0), (dict(max_pages=262144 // 32), 0), (dict(max_pages=262144 // 32 + 1), 3),
    (dict(num_kv_heads=256), 0), (dict(num_kv_heads=257), 3),
])
def test_the_eviction_workspace_of_what_eviction_serves(sa, change, status):  # noqa: F811
    n = ctypes.c_size_t()
    d = desc(sa, **change)
    assert sa._lib.sparse_attn_paged_evict_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status
    d.weights = None                               # the query needs no arrays but the cache's
    assert sa._lib.sparse_attn_paged_evict_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status


@pytest.mark.parametrize("change", [
    dict(max_tokens=300000), dict(max_tokens=262145), dict(num_kv_heads=257, keep=[64] * 257),
    dict(sinks=-1), dict(recent=-4), dict(keep=[64, 2**31]), dict(keep=[64, 19]), dict(keep=[64]),
])
def test_decode_layer_refuses_what_eviction_cannot_serve(sa, change):  # noqa: F811
    # before anything is allocated: nowhere near a device
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    args = dict(batch=1, num_q_heads=8, num_kv_heads=2, head_dim=64, page=16, num_pages=10,
                max_tokens=1000, keep=[64, 80], device="cpu")
    with pytest.raises(ValueError, match="keep|eviction|sinks"):
        PagedDecodeLayer(**{**args, **change})
    for kind in (dict(sinks=4.0), dict(recent="16")):
        with pytest.raises(TypeError):
            PagedDecodeLayer(**{**args, **kind})
    # budgets that no row can pass need no eviction: the first refusal is the device's
    for fine in (dict(max_tokens=262144), dict(max_tokens=300000, keep=[300000] * 2)):
        with pytest.raises(ValueError, match="CUDA device"):
            PagedDecodeLayer(**{**args, **fine})


@pytest.mark.parametrize("torch", [True, False])
def test_star_import_with_and_without_torch(sa, torch):  # noqa: F811
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("" if torch else "import sys; sys.modules['torch'] = None\n") + (
        "from head_heterogeneous_block_gb300 import *\n"
        f"assert callable(sparse_attn_paged_append) and ('PagedCache' in globals()) is {torch}\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_binding_functions_raise_on_a_refusal(sa):  # noqa: F811
    d = desc(sa)
    with pytest.raises(sa.SparseAttnError) as e:
        sa.sparse_attn_paged_append(d, P, P, (1024, 128, 4), (1024, 128, 256), 4, None, None, P, P,
                                    stream=0)
    assert e.value.status == 1
    with pytest.raises(sa.SparseAttnError) as e:
        sa.sparse_attn_paged_attend(d, P, 1024, 128, 7, P, None, None, P, 1 << 40, P,
                                    o_dtype=sa.SA_DTYPE_BF16, stream=0)
    assert e.value.status == 2
    with pytest.raises(sa.SparseAttnError) as e:
        sa.sparse_attn_paged_evict(d, [50, 19], 4, 16, P, P, P, P, 1 << 40, P, stream=0)
    assert e.value.status == 1
    for keep in ([50], [50, -1], [50, 2**31]):
        with pytest.raises(ValueError):
            sa.sparse_attn_paged_evict(d, keep, 4, 16, P, P, P, P, 1 << 40, P, stream=0)
