"""The paged cache without a GPU: the oracle's own pins, and the argument
checks of the C entry points and of PagedCache, which answer before anything
touches a device."""
import ctypes
import math

import numpy as np
import pytest

from oracle import paged as op


@pytest.fixture(scope="module")
def sa():
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa


# ---------------------------------------------------------------- oracle pins
def _pool(seed, pages, page, d):
    r = np.random.default_rng(seed)
    return r.standard_normal((pages, page, d)), r.standard_normal((pages, page, d))


def test_oracle_attend_equals_contiguous_attention():
    from oracle.attention import attend_all
    page, d = 16, 64
    k, v = _pool(0, 9, page, d)
    table = np.array([[[3, 7, 1, 8]]], np.int32)
    lens = np.array([[64]], np.int32)
    q = np.random.default_rng(1).standard_normal((1, 2, d))
    o, lse, w, absv, absqk = op.attend(q, k, v, table, lens, np.zeros((1, 1, 64)))
    kk, vv = k[table[0, 0]].reshape(-1, d), v[table[0, 0]].reshape(-1, d)
    # the last query row of one 64-token block sees every key
    full = np.zeros((2, 64, d))
    full[:, -1] = q[0]
    ref = attend_all(full, kk[None], vv[None], np.zeros((2, 1, 1), np.int32),
                     np.ones((2, 1), np.int32), 64)
    for h in range(2):
        np.testing.assert_allclose(o[0, h], ref[h][0][-1], rtol=1e-12)
        np.testing.assert_allclose(lse[0, h], ref[h][1][-1], rtol=1e-12)
    np.testing.assert_allclose(w.sum(), 2.0, rtol=1e-12)
    assert (absv >= np.abs(o) - 1e-15).all() and (absqk > 0).all()


def test_oracle_attend_of_an_empty_row():
    k, v = _pool(2, 3, 16, 64)
    q = np.ones((1, 1, 64))
    o, lse, w, _, _ = op.attend(q, k, v, np.full((1, 1, 1), -1, np.int32), np.zeros((1, 1), np.int32),
                                np.full((1, 1, 16), 0.5))
    assert (o == 0).all() and lse[0, 0] == -math.inf and (w == 0.5).all()


def test_oracle_kept_slots_by_hand():
    w = np.array([0.5, 0.1, 0.9, 0.9, 0.2, 0.9])
    p = np.arange(6)
    assert op.kept_slots(w, p, 3, 0, 0) == [2, 3, 5]
    assert op.kept_slots(w, p, 2, 0, 0) == [2, 3]              # ties: the lower slot
    assert op.kept_slots(w, p, 3, 1, 1) == [0, 2, 5]
    assert op.kept_slots(w, p[::-1].copy(), 3, 1, 1) == [0, 2, 5]
    assert op.kept_slots(np.array([math.nan, -math.inf, 1.0, -0.0, 0.0]), np.arange(5), 4, 0, 0) == [1, 2, 3, 4]
    assert op.kept_slots(w, p, 0, 0, 0) == []


def test_oracle_evict_moves_as_few_as_can_be():
    page, d = 16, 64
    k, v = _pool(3, 2, page, d)
    table, lens = np.array([[[1, 0]]], np.int32), np.array([[20]], np.int32)
    w = np.zeros((1, 1, 32))
    w[0, 0, [3, 17, 18, 5]] = 1.0
    pos = np.arange(32, dtype=np.int32)[None, None]
    k2, v2, lens2, w2, pos2 = op.evict(k, v, table, lens, w, pos, [4], 0, 1)
    # kept: 19 (recent), 3, 5 and 17; slot 3 stays, 5, 17, 19 fill slots 0, 1, 2
    assert lens2[0, 0] == 4
    assert pos2[0, 0, :4].tolist() == [5, 17, 19, 3]
    np.testing.assert_array_equal(k2[1, 0], k[1, 5])
    np.testing.assert_array_equal(k2[1, 1], k[0, 1])
    np.testing.assert_array_equal(v2[1, 2], v[0, 3])
    np.testing.assert_array_equal(k2[1, 3:], k[1, 3:])
    np.testing.assert_array_equal(k2[0], k[0])


# ---------------------------------------------------------------- refusals
P = 8192          # an aligned, non-null address that no call gets to use


def desc(sa, **kw):
    d = dict(k_pages=P, v_pages=P, table=P, lens=P, weights=P, positions=P, num_pages=40,
             k_page_stride=32 * 128, v_page_stride=32 * 128, page=32, max_pages=4, batch=2,
             num_kv_heads=2, head_dim=128)
    d.update(kw)
    return sa.PagedCacheDesc(**d)


BAD_DESC = [
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(page=0), 2), (dict(max_pages=0), 2), (dict(batch=0), 2), (dict(num_kv_heads=-1), 2),
    (dict(num_pages=0), 2), (dict(num_pages=1 << 31), 2), (dict(max_pages=1 << 30), 2),
    (dict(batch=1 << 24, num_kv_heads=2), 2), (dict(batch=1 << 12, max_pages=1 << 20), 2),
    (dict(head_dim=96), 3), (dict(head_dim=256), 3), (dict(page=8), 3), (dict(page=48), 3),
    (dict(page=512, k_page_stride=1 << 20, v_page_stride=1 << 20), 3),
    (dict(k_page_stride=32 * 128 - 8), 1), (dict(v_page_stride=32 * 128 + 4), 1),
    (dict(k_page_stride=1 << 38), 1), (dict(k_pages=P + 8), 1), (dict(v_pages=P + 2), 1),
    (dict(lens=P + 2), 1), (dict(weights=P + 1), 1),
]


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def _append(sa, d, k=P, v=P, ks=(1024, 128, 256), vs=(1024, 128, 256), n=4, counts=P, start=P,
            lens_out=P, status=P):
    return sa._lib.sparse_attn_paged_append(
        ctypes.byref(d) if d is not None else None, k, v, None if ks is None else _strides(*ks),
        None if vs is None else _strides(*vs), n, counts, start, lens_out, status, None)


def _attend(sa, d, q=P, qsb=1024, qsh=128, hq=8, o=P, dt=0, lse=P, w=None, ws=P, wsb=1 << 40, status=P):
    return sa._lib.sparse_attn_paged_attend(ctypes.byref(d) if d is not None else None, q, qsb, qsh,
                                            hq, o, dt, lse, w, ws, wsb, status, None)


def _evict(sa, d, keep=(50, 60), sinks=4, recent=16, lens=P, w=P, pos=P, ws=P, wsb=1 << 40, status=P):
    arr = None if keep is None else (ctypes.c_int32 * len(keep))(*keep)
    return sa._lib.sparse_attn_paged_evict(ctypes.byref(d) if d is not None else None, arr, sinks,
                                           recent, lens, w, pos, ws, wsb, status, None)


@pytest.mark.parametrize("change,status", BAD_DESC)
def test_bad_descriptors_are_refused_by_every_call(sa, change, status):
    d = desc(sa, **change)
    assert _append(sa, d) == status
    assert _attend(sa, d) == status
    assert _evict(sa, d) == status
    n = ctypes.c_size_t()
    assert sa._lib.sparse_attn_paged_attend_workspace_size(ctypes.byref(d), 8, 0, ctypes.byref(n)) == status
    assert sa._lib.sparse_attn_paged_evict_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status


def test_a_null_descriptor_is_refused(sa):
    n = ctypes.c_size_t()
    assert _append(sa, None) == 1 and _attend(sa, None) == 1 and _evict(sa, None) == 1
    assert sa._lib.sparse_attn_paged_evict_workspace_size(None, ctypes.byref(n)) == 1
    assert sa._lib.sparse_attn_paged_evict_workspace_size(ctypes.byref(desc(sa)), None) == 1
    assert sa._lib.sparse_attn_paged_attend_workspace_size(ctypes.byref(desc(sa)), 8, 0, None) == 1


@pytest.mark.parametrize("change,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(lens_out=None), 1), (dict(status=None), 1), (dict(k=P + 8), 1), (dict(v=P + 2), 1),
    (dict(counts=P + 2), 1), (dict(start=P + 1), 1), (dict(n=0), 2), (dict(n=-3), 2),
    (dict(ks=(1024, 128, 4)), 1), (dict(vs=(-8, 128, 8)), 1),
])
def test_append_refusals(sa, change, status):
    assert _append(sa, desc(sa), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(status=None), 1),
    (dict(q=P + 8), 1), (dict(o=P + 4), 1), (dict(ws=P + 64), 1), (dict(lse=P + 2), 1),
    (dict(dt=2), 1), (dict(dt=-1), 1), (dict(hq=7), 2), (dict(hq=0), 2), (dict(hq=-2), 2),
    (dict(hq=2 * 1025), 2), (dict(qsb=1020), 1), (dict(qsb=0), 1), (dict(qsh=64), 1),
    (dict(qsh=1 << 38), 1),
])
def test_attend_refusals(sa, change, status):
    assert _attend(sa, desc(sa), **change) == status


def test_attend_needs_weights_to_accumulate(sa):
    assert _attend(sa, desc(sa, weights=None), w=P) == 1
    n = ctypes.c_size_t()
    assert sa._lib.sparse_attn_paged_attend_workspace_size(ctypes.byref(desc(sa)), 8, 2,
                                                           ctypes.byref(n)) == 1
    assert sa._lib.sparse_attn_paged_attend_workspace_size(ctypes.byref(desc(sa)), 7, 1,
                                                           ctypes.byref(n)) == 2


@pytest.mark.parametrize("change,status", [
    (dict(keep=None), 1), (dict(lens=None), 1), (dict(w=None), 1), (dict(ws=None), 1),
    (dict(status=None), 1), (dict(pos=None), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1),
    (dict(keep=(50, 19)), 1), (dict(keep=(-1, 50), sinks=0, recent=0), 1),
    (dict(sinks=2**31 - 1, recent=2**31 - 1), 1), (dict(ws=P + 8), 1), (dict(w=P + 2), 1),
    (dict(wsb=0), 1),
])
def test_evict_refusals(sa, change, status):
    assert _evict(sa, desc(sa), **change) == status


def test_evict_refuses_what_the_cache_does_not_hold(sa):
    assert _evict(sa, desc(sa, weights=None)) == 1
    assert _evict(sa, desc(sa, positions=None)) == 1           # positions_out without positions
    assert _evict(sa, desc(sa, max_pages=262144 // 32 + 1)) == 3
    assert _evict(sa, desc(sa, num_kv_heads=257), keep=[50] * 257) == 3


def test_python_class_refuses_cpu_tensors_and_wrong_types(sa):
    import torch
    k = torch.zeros(4, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, 2, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sa.PagedCache(k, k, table, lens)
    with pytest.raises(TypeError):
        sa.PagedCache(k.half(), k, table, lens)
    with pytest.raises(TypeError):
        sa.PagedCache(k, k, table.long(), lens)
    with pytest.raises(AttributeError):
        sa.no_such_name


# ---------------------------------------------------------------- the page book
def test_page_book_hands_out_and_takes_back(sa):
    from head_heterogeneous_block_gb300.paged import PageBook
    book = PageBook(num_pages=7, page=16, batch=2, num_kv_heads=2, max_pages=3)
    assert book.grow([17, 0]) == [(0, 0, 0, 0), (0, 0, 1, 1), (0, 1, 0, 2), (0, 1, 1, 3)]
    assert book.lens == [[17, 17], [0, 0]] and len(book.free) == 3
    assert book.grow([0, 16]) == [(1, 0, 0, 4), (1, 1, 0, 5)]
    with pytest.raises(MemoryError):
        book.grow([0, 1])                       # two pages, one free
    assert book.lens == [[17, 17], [16, 16]] and len(book.free) == 1
    with pytest.raises(ValueError):
        book.grow([32, 0])                      # past the table
    book.shrink(0, [16, 40])
    assert book.lens == [[16, 17], [16, 16]] and sorted(book.free) == [1, 6]
    assert book.grow([0, 1]) == [(1, 0, 1, 1), (1, 1, 1, 6)]
    book.shrink(1, [0, 0])
    assert book.rows[1] == [[], []] and sorted(book.free) == [1, 4, 5, 6]


@pytest.mark.parametrize("seed", range(4))
def test_page_book_never_shares_a_page(sa, seed):
    from head_heterogeneous_block_gb300.paged import PageBook
    r = np.random.default_rng(seed)
    book = PageBook(num_pages=60, page=16, batch=3, num_kv_heads=2, max_pages=12)
    table = {}
    for _ in range(200):
        if r.random() < 0.7:
            try:
                for b, g, e, p in book.grow([int(x) for x in r.integers(0, 20, 3)]):
                    table[b, g, e] = p
            except (MemoryError, ValueError):
                pass
        else:
            book.shrink(int(r.integers(0, 3)), [int(x) for x in r.integers(0, 150, 2)])
        owned = [p for rows in book.rows for row in rows for p in row]
        assert sorted(owned + book.free) == list(range(60))
        for b in range(3):
            for g in range(2):
                assert len(book.rows[b][g]) == -(-book.lens[b][g] // 16)
                assert [table[b, g, e] for e in range(len(book.rows[b][g]))] == book.rows[b][g]
