"""Objects made behind a long queue of one stream, used at once on another."""
import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402
from tests.test_gpu_packed import run, sa  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def busy():
    """Some tenths of a second of the current stream."""
    torch.cuda._sleep(400_000_000)


def test_a_pool(sa):  # noqa: F811
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.full((2, 2, 8), -1, **i32), torch.zeros(2, 2, **i32)
    slots, counts = torch.zeros(2, 100, dtype=torch.int64, device="cuda"), torch.tensor([50, 33], **i32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    pool = sa.PagePool(table, lens, 16, num_pages=40)
    pool.grow(slots, counts=counts, stream=side)
    side.synchronize()
    assert lens.tolist() == [[50, 50], [33, 33]] and pool.owned.tolist() == [[4, 4], [3, 3]]
    assert int(pool.free_count) == 40 - 14 and table[0, 0, :4].tolist() == [0, 1, 2, 3]
    assert int(pool.dev_status.item()) == 0


def test_the_pool_of_a_cache(sa):  # noqa: F811
    i32 = dict(dtype=torch.int32, device="cuda")
    pools = [torch.zeros(40, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = sa.PagedCache(*pools, torch.zeros(2, 2, 8, **i32), torch.full((2, 2), 77, **i32))
    slots = torch.zeros(2, 100, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    pool = sa.PagePool.of(cache)
    pool.grow(slots, stream=side)
    side.synchronize()
    assert cache.lens.tolist() == [[50, 50], [50, 50]] and int(pool.dev_status.item()) == 0


def test_attention_and_rotary_positions(sa):  # noqa: F811
    q, k, v, cq, ck = tp.inputs(120, [700, 40], [3000, 40], 8, 2, 64, device="cuda")
    want = run(sa, 8, 2, 64, q, k, v, cq, ck)[0]
    pos = torch.arange(740, dtype=torch.int32, device="cuda")
    turned = sa.Rotary(64)(q, k[:740], pos)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.full((1 << 26,), 0x7f, dtype=torch.uint8, device="cuda")
    busy()
    junk.fill_(0x7e)                     # still to be written where its memory is handed out again
    del junk
    att, rot = sa.PackedAttention(8, 2, 64, tokens=740, keys=3040, batch=2), sa.Rotary(64)
    out = att(q, k, v, cq, ck, stream=side)
    got = rot(q, k[:740], pos, stream=side)[0]
    side.synchronize()
    torch.cuda.synchronize()
    tp.same(out, want)
    tp.same(got, turned)
    assert int(att.dev_status.item()) == 0 and int(rot.dev_status.item()) == 0
