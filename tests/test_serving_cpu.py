"""The operators that take prompts into a paged cache without a GPU: the oracles'
own pins, and the argument checks of the C entry points and classes, which
answer before anything touches a device."""
import ctypes
import math

import numpy as np
import pytest

from oracle import packed as opk
from oracle import pages as opg
from oracle import rotary as orot


@pytest.fixture(scope="module")
def sa():
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa


# ---------------------------------------------------------------- oracle pins
def test_oracle_packed_equals_block_attention():
    from oracle.attention import attend_all
    r = np.random.default_rng(0)
    S, d, B = 128, 16, 64
    q, k, v = (r.standard_normal((S, h, d)) for h in (2, 1, 1))
    o, lse, _, _ = opk.attend(q, k, v, [0, S], [0, S])
    idx = np.zeros((2, 2, 2), np.int32)
    idx[:, 1] = [0, 1]
    cnt = np.array([[1, 2], [1, 2]], np.int32)
    ref = attend_all(q.transpose(1, 0, 2), k.transpose(1, 0, 2), v.transpose(1, 0, 2), idx, cnt, B)
    # two orders of a sum of up to 128 products of at most 8: 128 * 8 * 2^-53 < 1e-12, however small the sum
    for item, (ro, rl) in ref.items():
        h, i = divmod(item, 2)
        np.testing.assert_allclose(o[i * B:(i + 1) * B, h], ro, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(lse[i * B:(i + 1) * B, h], rl, rtol=1e-12, atol=1e-12)


def test_oracle_packed_chunks_and_rows_without_keys():
    r = np.random.default_rng(1)
    q, k, v = (r.standard_normal((9, h, 8)) for h in (2, 1, 1))
    whole, lse, _, _ = opk.attend(q, k, v, [0, 9], [0, 9])
    part, plse, _, _ = opk.attend(q[6:], k, v, [0, 3], [0, 9])       # the last three tokens as a chunk
    np.testing.assert_allclose(part, whole[6:], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(plse, lse[6:], rtol=1e-12, atol=1e-12)
    o, l, _, _ = opk.attend(q[:4], k, v, [0, 4], [0, 2])             # two queries see nothing
    assert (o[:2] == 0).all() and (l[:2] == -math.inf).all() and np.isfinite(l[2:]).all()
    o, _, _, _ = opk.attend(q, k, v, [2, 3], [0, 1])
    assert np.isnan(o[:2]).all() and np.isnan(o[3:]).all()


def test_oracle_rotary_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    f = [math.pi / 2, 0.0]
    np.testing.assert_allclose(orot.rotate(x, [1], f), [[[-3.0, 2.0, 1.0, 4.0, 9.0]]], atol=1e-15)
    np.testing.assert_allclose(orot.rotate(x, [1], f, 2.0, True), [[[-4.0, 2.0, 6.0, 8.0, 9.0]]], atol=1e-15)
    # scores depend on the distance alone
    r = np.random.default_rng(2)
    q, k = r.standard_normal((2, 1, 1, 8))
    g = [1.0, 0.3, 0.07, 0.01]
    a = [float((orot.rotate(q, [p + 5], g) * orot.rotate(k, [p], g)).sum()) for p in (0, 3, 1000)]
    np.testing.assert_allclose(a, a[0], rtol=1e-9)


def test_oracle_pages_by_hand():
    table = np.full((2, 1, 4), -1)
    table[1, 0, :3] = [5, 6, 7]
    out = opg.grow(table, np.array([[0], [20]]), np.array([[0], [3]]), [1, 2], 16, [(0, 20), (20, 21)],
                   start=[100, 7], tokens=22)
    # row 1 needs two of its three pages: page 7 comes back, above 1 and 2, and goes out first
    assert out["table"][0, 0].tolist() == [7, 2, -1, -1] and out["free"] == [1]
    assert out["owned"].tolist() == [[2], [2]] and out["lens"].tolist() == [[20], [21]]
    assert out["slots"][0, [0, 15, 16, 20, 21]].tolist() == [112, 127, 32, 6 * 16 + 4, -1]
    assert out["token_positions"][[0, 19, 20, 21]].tolist() == [100, 119, 7, 0]


# ---------------------------------------------------------------- frequencies
def test_rotary_frequencies(sa):
    from head_heterogeneous_block_gb300.rotary import rotary_frequencies as rf
    f, m = rf(8, 10000.0)
    np.testing.assert_allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-12)
    assert m == 1.0
    np.testing.assert_allclose(rf(8, 10000.0, {"type": "linear", "factor": 4})[0], [x / 4 for x in f], rtol=1e-12)
    g = rf(8, 10000.0, {"type": "ntk", "factor": 4})[0]
    assert g[0] == 1.0
    np.testing.assert_allclose(g[3], f[3] / 4, rtol=1e-12)
    # turns over 1000 positions: 159, 15.9, 1.59, 0.159
    g = rf(8, 10000.0, {"type": "wavelength", "factor": 8, "low": 1, "high": 4, "original": 1000})[0]
    x = (0.01 * 1000 / (2 * math.pi) - 1) / 3
    np.testing.assert_allclose(g, [1.0, 0.1, 0.01 * x + 0.01 / 8 * (1 - x), 0.001 / 8], rtol=1e-12)
    g, m = rf(64, 10000.0, {"type": "yarn", "factor": 4, "original": 4096})
    f = rf(64, 10000.0)[0]
    lo = math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000)))
    hi = math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000)))
    assert g[:lo + 1] == f[:lo + 1] and lo < hi < 32
    np.testing.assert_allclose(g[hi:], [x / 4 for x in f[hi:]], rtol=1e-12)
    mid = (lo + hi) // 2
    t = (mid - lo) / (hi - lo)
    np.testing.assert_allclose(g[mid], f[mid] * (1 - t) + f[mid] / 4 * t, rtol=1e-12)
    np.testing.assert_allclose(m, 0.1 * math.log(4) + 1, rtol=1e-12)


@pytest.mark.parametrize("rot,base,scaling", [
    (7, 1e4, None), (0, 1e4, None), (8, 1.0, None), (8, -3.0, None), (8, float("inf"), None),
    (8, 1e4, {"type": "cubic", "factor": 2}), (8, 1e4, {"type": "linear"}), (8, 1e4, {"type": "linear", "factor": 0}),
    (8, 1e4, {"type": "linear", "factor": 2, "low": 1}), (8, 1e4, {"type": "ntk", "factor": float("nan")}),
    (8, 1e4, {"type": "wavelength", "factor": 2, "low": 4, "high": 1, "original": 100}),
    (8, 1e4, {"type": "yarn", "factor": 2, "original": 100, "beta_fast": 1, "beta_slow": 2}), (8, 1e4, {"factor": 2}),
])
def test_rotary_frequencies_refusals(sa, rot, base, scaling):
    from head_heterogeneous_block_gb300.rotary import rotary_frequencies as rf
    with pytest.raises(ValueError):
        rf(rot, base, scaling)


# ---------------------------------------------------------------- refusals of the C entry points
P = 1 << 20                                     # an aligned address that nothing reads


def _packed_shape(sa, **kw):
    args = dict(q_stride_t=1024, q_stride_h=128, k_stride_t=256, k_stride_h=128, v_stride_t=256, v_stride_h=128,
                o_stride_t=1024, o_stride_h=128, total_q=100, total_k=100, batch=3, num_q_heads=8, num_kv_heads=2,
                head_dim=128, scale=0.1)
    args.update(kw)
    return sa.PackedShape(**args)


def _packed(sa, s, q=P, k=2 * P, v=3 * P, cu_q=P, cu_k=P, o=4 * P, lse=P, ws=P, wsb=1 << 40, status=P):
    return sa._lib.sparse_attn_packed_forward(ctypes.byref(s) if s is not None else None, q, k, v, cu_q, cu_k, o, lse,
                                              ws, wsb, status, None)


@pytest.mark.parametrize("change,status", [
    (dict(total_q=-1), 2), (dict(total_k=-1), 2), (dict(total_q=(1 << 30) + 1), 2), (dict(batch=0), 2),
    (dict(batch=(1 << 20) + 1), 2), (dict(num_q_heads=0), 2), (dict(num_kv_heads=0), 2), (dict(num_kv_heads=3), 2),
    (dict(num_q_heads=1 << 22, num_kv_heads=1 << 22), 2), (dict(head_dim=96), 3), (dict(head_dim=256), 3),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
])
def test_packed_shapes_are_refused_by_both_calls(sa, change, status):
    s = _packed_shape(sa, **change)
    assert _packed(sa, s) == status
    n = ctypes.c_size_t()
    assert sa._lib.sparse_attn_packed_workspace_size(ctypes.byref(s), ctypes.byref(n)) == status


@pytest.mark.parametrize("change", [
    dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(cu_q=None), dict(cu_k=None), dict(ws=None),
    dict(status=None), dict(q=P + 8), dict(k=P + 2), dict(v=P + 8), dict(o=P + 8), dict(cu_q=P + 2), dict(cu_k=P + 1),
    dict(lse=P + 2), dict(ws=P + 128), dict(o=P), dict(o=2 * P), dict(o=3 * P)])
def test_packed_refusals(sa, change):
    assert _packed(sa, _packed_shape(sa), **change) == 1


@pytest.mark.parametrize("change", [
    dict(q_stride_t=1020), dict(q_stride_h=64), dict(k_stride_t=0), dict(k_stride_h=0), dict(v_stride_t=-256),
    dict(v_stride_h=1 << 38), dict(o_stride_t=128), dict(o_stride_h=1024, o_stride_t=1032)])
def test_packed_strides(sa, change):
    assert _packed(sa, _packed_shape(sa, **change)) == 1


def test_packed_null_shape(sa):
    n = ctypes.c_size_t()
    assert _packed(sa, None) == 1
    assert sa._lib.sparse_attn_packed_workspace_size(None, ctypes.byref(n)) == 1
    assert sa._lib.sparse_attn_packed_workspace_size(ctypes.byref(_packed_shape(sa)), None) == 1


def _rot(sa, **kw):
    args = dict(turns=P, factor=1.0, head_dim=128, rot_dim=64, interleaved=0)
    args.update(kw)
    return sa.RotaryDesc(**args)


def _s2(s):
    return None if s is None else (ctypes.c_int64 * 2)(*s)


def _rotary(sa, r, tokens=4, hq=8, hkv=2, pos=P, q=P, qs=(1024, 128), k=2 * P, ks=(256, 128), qo=3 * P, qos=(1024, 128),
            ko=4 * P, kos=(256, 128)):
    return sa._lib.sparse_attn_rotary(ctypes.byref(r) if r is not None else None, tokens, hq, hkv, pos, q, _s2(qs), k,
                                      _s2(ks), qo, _s2(qos), ko, _s2(kos), None)


def _desc(sa, **kw):
    args = dict(k_pages=P, v_pages=P, table=P, lens=P, weights=P, positions=P, num_pages=10, k_page_stride=32 * 128,
                v_page_stride=32 * 128, page=32, max_pages=4, batch=2, num_kv_heads=2, head_dim=128)
    args.update(kw)
    return sa.PagedCacheDesc(**args)


def _store(sa, r, cache, tokens=4, hq=8, pos=P, q=P, qs=(1024, 128), k=2 * P, ks=(256, 128), v=5 * P, vs=(256, 128),
           qo=3 * P, qos=(1024, 128), ko=4 * P, kos=(256, 128), slots=P, status=P):
    return sa._lib.sparse_attn_rotary_store(ctypes.byref(r) if r is not None else None, tokens, hq, pos, q, _s2(qs), k,
                                            _s2(ks), v, _s2(vs), qo, _s2(qos), ko, _s2(kos),
                                            ctypes.byref(cache) if cache is not None else None, slots, status, None)


@pytest.mark.parametrize("change,status", [
    (dict(turns=None), 1), (dict(turns=P + 4), 1), (dict(factor=float("nan")), 1), (dict(factor=float("inf")), 1),
    (dict(interleaved=2), 1), (dict(head_dim=96), 3), (dict(rot_dim=8), 3), (dict(rot_dim=24), 3), (dict(rot_dim=144), 3),
    (dict(rot_dim=0), 3)])
def test_rotary_descriptors(sa, change, status):
    assert _rotary(sa, _rot(sa, **change)) == status
    assert _store(sa, _rot(sa, **change), _desc(sa)) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 2), (dict(tokens=(1 << 30) + 1), 2), (dict(hq=0), 2), (dict(hkv=0), 2), (dict(pos=None), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(qs=None), 1), (dict(ks=None), 1),
    (dict(qos=None), 1), (dict(kos=None), 1), (dict(q=P + 8), 1), (dict(k=P + 2), 1), (dict(qo=P + 8), 1),
    (dict(ko=P + 4), 1), (dict(pos=P + 2), 1), (dict(qs=(1020, 128)), 1), (dict(ks=(-256, 128)), 1),
    (dict(qos=(1024, 64)), 1), (dict(kos=(0, 128)), 1), (dict(qos=(1 << 38, 128)), 1),
    (dict(qo=P, qos=(2048, 128)), 1), (dict(ko=2 * P, kos=(512, 128)), 1), (dict(qo=2 * P), 1), (dict(ko=P), 1),
    (dict(qo=4 * P), 1)])
def test_rotary_refusals(sa, change, status):
    assert _rotary(sa, _rot(sa), **change) == status


@pytest.mark.parametrize("change", [dict(v=None), dict(slots=None), dict(status=None), dict(vs=None), dict(v=P + 8),
                                    dict(slots=P + 4), dict(status=P + 2), dict(vs=(252, 128)), dict(vs=(-8, 128)),
                                    dict(kos=None)])
def test_rotary_store_refusals(sa, change):
    assert _store(sa, _rot(sa), _desc(sa), **change) == 1


def test_rotary_store_refuses_bad_caches(sa):
    assert _store(sa, _rot(sa), None) == 1 and _store(sa, None, _desc(sa)) == 1 and _rotary(sa, None) == 1
    assert _store(sa, _rot(sa), _desc(sa, head_dim=64)) == 2
    assert _store(sa, _rot(sa), _desc(sa, page=48)) == 3
    assert _store(sa, _rot(sa), _desc(sa, k_pages=None)) == 1


def _pool(sa, **kw):
    args = dict(table=P, lens=P, owned=P, free_pages=P, free_count=P, weights=P, positions=P, num_pages=100, page=32,
                max_pages=4, batch=2, num_kv_heads=2)
    args.update(kw)
    return sa.PagePoolDesc(**args)


def _grow(sa, pool, ws=P, wsb=1 << 40, status=P, growth=True, **kw):
    args = dict(cu=P, counts=P, ended=P, start=P, slots=8 * P, token_positions=16 * P, granted=P, lens_out=P, owned_out=P,
                free_count_out=P, start_out=P, tokens=10)
    args.update(kw)
    g = sa.PageGrowth(**args)
    return sa._lib.sparse_attn_paged_grow(ctypes.byref(pool) if pool is not None else None,
                                          ctypes.byref(g) if growth else None, ws, wsb, status, None)


@pytest.mark.parametrize("change,status", [
    (dict(table=None), 1), (dict(lens=None), 1), (dict(owned=None), 1), (dict(free_pages=None), 1),
    (dict(free_count=None), 1), (dict(table=P + 2), 1), (dict(weights=P + 1), 1), (dict(positions=P + 2), 1),
    (dict(num_pages=0), 2), (dict(num_pages=1 << 30), 2), (dict(page=0), 2), (dict(max_pages=0), 2), (dict(batch=0), 2),
    (dict(num_kv_heads=-1), 2), (dict(batch=1 << 20, num_kv_heads=2), 2), (dict(max_pages=1 << 26), 2),
    (dict(page=16, max_pages=1 << 26, batch=16, num_kv_heads=2), 2), (dict(page=8), 3), (dict(page=48), 3),
    (dict(page=512), 3)])
def test_pools_are_refused_by_both_calls(sa, change, status):
    assert _grow(sa, _pool(sa, **change)) == status
    n = ctypes.c_size_t()
    assert sa._lib.sparse_attn_paged_grow_workspace_size(ctypes.byref(_pool(sa, **change)), ctypes.byref(n)) == status


@pytest.mark.parametrize("change,status", [
    (dict(slots=None), 1), (dict(lens_out=None), 1), (dict(owned_out=None), 1), (dict(free_count_out=None), 1),
    (dict(ws=None), 1), (dict(status=None), 1), (dict(ws=P + 64), 1), (dict(wsb=100), 1), (dict(slots=8 * P + 4), 1),
    (dict(slots=P), 1), (dict(slots=16 * P), 1), (dict(token_positions=P), 1), (dict(token_positions=8 * P + 40), 1),
    (dict(cu=P + 2), 1), (dict(granted=P + 1), 1), (dict(growth=False), 1), (dict(tokens=-1), 2),
    (dict(tokens=11, cu=None), 2), (dict(tokens=(1 << 30) + 1), 2)])
def test_grow_refusals(sa, change, status):
    assert _grow(sa, _pool(sa), **change) == status


def test_grow_workspace(sa):
    n = ctypes.c_size_t()
    assert _grow(sa, None) == 1
    assert sa._lib.sparse_attn_paged_grow_workspace_size(ctypes.byref(_pool(sa)), None) == 1
    assert sa._lib.sparse_attn_paged_grow_workspace_size(ctypes.byref(_pool(sa)), ctypes.byref(n)) == 0
    assert n.value >= 4 * 16


# ---------------------------------------------------------------- refusals of the classes
def test_classes_refuse_other_devices_and_sizes(sa):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        sa.PackedAttention(8, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        sa.Rotary(128, device="cpu")
    for kw in (dict(head_dim=96), dict(head_dim=128, rot_dim=24), dict(head_dim=64, rot_dim=128)):
        with pytest.raises(ValueError):
            sa.Rotary(**kw)
    with pytest.raises(ValueError):
        sa.PagePool(torch.zeros(1, 1, 2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), 16, num_pages=4)


def test_native_calls_check_their_tensors(sa):
    torch = pytest.importorskip("torch")
    from head_heterogeneous_block_gb300._device import calls
    q, k = torch.zeros(4, 8, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16()
    cu = torch.tensor([0, 4], dtype=torch.int32)

    def packed(q=q, k=k, v=k, cu_q=cu, cu_k=None, out=q, lse=None, heads=8):
        return calls.packed(0, heads, 2, 64, 0.125, 100, 4, 100, q, k, v, cu_q, cu_k, out, lse, P, 1 << 40, P, 0)

    for kw in (dict(q=q.float()), dict(q=q.half()), dict(q=3), dict(q=None)):
        with pytest.raises(TypeError):
            packed(**kw)
    for kw in (dict(), dict(q=q[0]), dict(q=q[:, :3]), dict(q=q[..., ::2]), dict(heads=7)):
        with pytest.raises(ValueError):
            packed(**kw)                        # CPU tensors, at the latest
    with pytest.raises(TypeError):
        calls.packed(1, 2, 3)
    with pytest.raises(TypeError):
        calls.packed("x", *range(18))
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        calls.rotary(P, 0, 64, q.float(), k, pos, q, k, 0)
    with pytest.raises(ValueError):
        calls.rotary(P, 0, 64, q, k, pos, q, k, 0)
    with pytest.raises(ValueError):
        calls.rotary_store(P, 0, 64, 2, q, k, k, pos, P, torch.zeros(2, 4, dtype=torch.int64), q, None, P, 0)
    pool = _pool(sa)
    at = ctypes.addressof(pool)
    slots = torch.zeros(2, 4, dtype=torch.int64)
    none = [None] * 10
    with pytest.raises(TypeError):
        calls.grow(at, 0, None, *none, P, 1 << 40, P, 0)
    for s in (slots, slots[0], torch.zeros(2, 3, dtype=torch.int64), slots.int(), torch.zeros(3, 4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            calls.grow(at, 0, s, *none, P, 1 << 40, P, 0)
