"""The binding's functions for pages, rotary positions and packed attention, on
addresses and explicit strides, against the classes: the same bits."""
import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402
from tests.test_gpu_packed import sa  # noqa: E402, F401
from tests.test_gpu_pages import state, to_gpu  # noqa: E402

pytestmark = pytest.mark.gpu


def workspace(need):
    return torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens_q,lens_k", [([200, 77], [200, 77]), ([20, 5], [4000, 300])])
@pytest.mark.parametrize("with_lse", [False, True])
def test_packed(sa, with_lse, lens_q, lens_k):  # noqa: F811
    q, k, v, cq, ck = tp.inputs(100, lens_q, lens_k, 8, 2, 64, device="cuda")
    fused = torch.cat((q, q), 1)[:, 3:11]
    att = sa.PackedAttention(8, 2, 64)
    lse = [torch.zeros(q.shape[:2], device="cuda") if with_lse else None for _ in range(2)]
    want = att(fused, k, v, cq, ck, lse=lse[0])
    out, status = torch.empty_like(q), status_word()
    s = sa.PackedShape(*fused.stride()[:2], *k.stride()[:2], *v.stride()[:2], *out.stride()[:2], q.shape[0], k.shape[0],
                       len(lens_q), 8, 2, 64, 64 ** -0.5)
    need = sa.sparse_attn_packed_workspace_size(s)
    ws = workspace(need)
    sa.sparse_attn_packed_forward(s, fused.data_ptr(), k.data_ptr(), v.data_ptr(), cq, ck, out.data_ptr(), lse[1], ws,
                                  need, status, stream=torch.cuda.current_stream())
    tp.same(out, want)
    if with_lse:
        tp.same(lse[1], lse[0])
    assert int(status.item()) == 0


def test_rotary(sa):  # noqa: F811
    r = sa.Rotary(64, rot_dim=32, interleaved=True, base=500000.0)
    qkv = torch.randn(50, 12, 64, device="cuda").bfloat16()
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    pos = torch.randint(0, 9999, (50,), dtype=torch.int32, device="cuda")
    want = r(q, k, pos)
    qo, ko = torch.empty_like(want[0]), torch.empty_like(want[1])
    desc = sa.RotaryDesc(r.turns.data_ptr(), r.factor, 64, 32, 1)
    sa.sparse_attn_rotary(desc, 50, 8, 2, pos, q.data_ptr(), q.stride()[:2], k.data_ptr(), k.stride()[:2], qo.data_ptr(),
                          qo.stride()[:2], ko.data_ptr(), ko.stride()[:2])
    tp.same(qo, want[0])
    tp.same(ko, want[1])
    # with the store: the cache's copy and k_out, or the cache's alone
    slots = torch.randperm(8 * 16, device="cuda")[:100].view(2, 50).contiguous()
    pools, status = [], status_word()
    for binding in (False, True):
        for with_k in (True, False):
            kp, vp = (torch.zeros(8, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            cache = sa.PagedCache(kp, vp, torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda"),
                                  torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
            ko = torch.zeros_like(want[1]) if with_k else None
            qo = torch.zeros_like(want[0])
            if binding:
                sa.sparse_attn_rotary_store(desc, 50, 8, pos, q.data_ptr(), q.stride()[:2], k.data_ptr(), k.stride()[:2],
                                            v.data_ptr(), v.stride()[:2], qo.data_ptr(), qo.stride()[:2],
                                            ko.data_ptr() if with_k else None, ko.stride()[:2] if with_k else None,
                                            cache.desc, slots, status)
            else:
                r.store(q, k, v, pos, cache, slots, q_out=qo, k_out=ko)
            tp.same(qo, want[0])
            if with_k:
                tp.same(ko, want[1])
            pools.append((kp, vp))
    for kp, vp in pools[1:]:
        tp.same(kp, pools[0][0])
        tp.same(vp, pools[0][1])
    assert int(status.item()) == 0 and (pools[0][0] != 0).any()


def test_grow(sa):  # noqa: F811
    s = state(101, 5, 3, 16, 30, 200, spare=4, free=300, extra=True)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, start0 = torch.tensor([0, 10, 10, 60, 61, 90], **i32), torch.arange(5, **i32) * 100
    ended = torch.tensor([False, True, False, False, True], device="cuda")
    got = []
    for binding in (False, True):
        d, pool = to_gpu(sa, s)
        slots = torch.zeros(3, 93, dtype=torch.int64, device="cuda")
        pos, granted, start = torch.zeros(93, **i32), torch.zeros(5, **i32), start0.clone()
        if binding:
            status = status_word()
            p = sa.PagePoolDesc(*(d[n].data_ptr() for n in ("table", "lens", "owned", "free_pages", "free_count", "weights",
                                                            "positions")), s["pages"], 16, 30, 5, 3)
            g = sa.PageGrowth(cu.data_ptr(), None, ended.data_ptr(), start.data_ptr(), slots.data_ptr(), pos.data_ptr(),
                              granted.data_ptr(), d["lens"].data_ptr(), d["owned"].data_ptr(), d["free_count"].data_ptr(),
                              start.data_ptr(), 93)
            need = sa.sparse_attn_paged_grow_workspace_size(p)
            ws = workspace(need)
            sa.sparse_attn_paged_grow(p, g, ws, need, status)
            assert int(status.item()) == 0
        else:
            pool.grow(slots, cu=cu, ended=ended, start=start, positions=pos, granted=granted)
            assert int(pool.dev_status.item()) == 0
        got.append([slots, pos, granted, start, *d.values()])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][2].tolist() == [10, 0, 50, 1, 29]
