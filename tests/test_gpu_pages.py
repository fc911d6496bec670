"""Pages and slots made on the GPU against the oracle: whole numbers, equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import pages as opg  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa


def state(seed, b, h, page, max_pages, held, spare=0, free=0, extra=False):
    """A consistent random state; rows hold up to `held` tokens, own up to `spare` pages more than they need."""
    r = np.random.default_rng(seed)
    lens = r.integers(0, held + 1, (b, h)) if spare else np.repeat(r.integers(0, held + 1, (b, 1)), h, 1)
    owned = np.minimum(max_pages, -(-lens // page) + (r.integers(0, spare + 1, (b, h)) if spare else 0))
    total = int(owned.sum()) + free + 2
    perm = r.permutation(total)
    table = np.full((b, h, max_pages), -1)
    mine = np.arange(max_pages) < owned[..., None]
    table[mine] = perm[:int(owned.sum())]
    s = {"table": table, "lens": lens, "owned": owned, "free": perm[int(owned.sum()):int(owned.sum()) + free].tolist(),
         "pages": total, "page": page}
    if extra:
        s["weights"] = r.random((b, h, max_pages * page)).astype(np.float32)
        s["positions"] = r.integers(0, 999, (b, h, max_pages * page))
    return s


def to_gpu(sa, s):
    d = {k: torch.tensor(s[k], dtype=torch.int32, device="cuda") for k in ("table", "lens", "owned")}
    d["free_pages"] = torch.full((s["pages"],), -7, dtype=torch.int32, device="cuda")
    d["free_pages"][:len(s["free"])] = torch.tensor(s["free"], dtype=torch.int32)
    d["free_count"] = torch.tensor([len(s["free"])], dtype=torch.int32, device="cuda")
    for k, t in (("weights", torch.float32), ("positions", torch.int32)):
        d[k] = torch.tensor(s[k], dtype=t, device="cuda") if k in s else None
    pool = sa.PagePool(d["table"], d["lens"], s["page"], free_pages=d["free_pages"], free_count=d["free_count"],
                       owned=d["owned"], weights=d["weights"], positions=d["positions"])
    return d, pool


def run(sa, s, spans, tokens, counts=None, ended=None, start=None, cu=True, status=0):
    d, pool = to_gpu(sa, s)
    b, h = s["lens"].shape
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = torch.full((h, tokens), 5, dtype=torch.int64, device="cuda")
    pos, granted = torch.full((tokens,), 5, **i32), torch.full((b,), 5, **i32)
    t = lambda x: None if x is None else torch.tensor(x, **i32)  # noqa: E731
    start_t = t(start)
    pool.grow(slots, cu=t([spans[0][0]] + [e for _, e in spans]) if cu else None, counts=t(counts),
              ended=None if ended is None else torch.tensor(ended, device="cuda"), start=start_t, positions=pos,
              granted=granted)
    torch.cuda.synchronize()
    assert int(pool.dev_status.item()) == status
    ref = opg.grow(s["table"], s["lens"], s["owned"], s["free"], s["page"], spans, counts, ended, start, tokens,
                   s.get("weights"), s.get("positions"))
    eq = lambda a, x: np.testing.assert_array_equal(a.cpu().numpy(), x)  # noqa: E731
    eq(slots, ref["slots"])
    eq(pos, ref["token_positions"])
    eq(granted, ref["granted"])
    eq(d["lens"], ref["lens"])
    eq(d["owned"], ref["owned"])
    eq(d["table"], ref["table"])
    assert int(d["free_count"]) == len(ref["free"])
    eq(d["free_pages"][:len(ref["free"])], ref["free"])
    if start is not None:
        eq(start_t, ref["start"])
    for k in ("weights", "positions"):
        if k in s:
            eq(d[k], ref[k])
    return d, pool, ref


def spans_of(counts, gap=0):
    ends = np.cumsum(np.asarray(counts) + gap)
    return [(int(e - c - gap), int(e)) for e, c in zip(ends, counts)]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("b,h", [(1, 1), (3, 2), (64, 8), (200, 4)])
def test_a_decode_step(sa, b, h, page):
    s = state(1, b, h, page, 10, 9 * page, free=b * h, extra=True)
    run(sa, s, [(x, x + 1) for x in range(b)], b, start=list(range(100, 100 + b)))
    run(sa, s, [(x, x + 1) for x in range(b)], b, cu=False)
    counts = [x % 2 for x in range(b)]
    run(sa, s, [(x, x + 1) for x in range(b)], b, counts=counts, cu=False)


@pytest.mark.parametrize("b,h,page,most", [(1, 8, 64, 40000), (5, 2, 16, 700), (16, 4, 32, 3000), (300, 16, 16, 20)])
def test_prompts_into_empty_rows(sa, b, h, page, most):
    r = np.random.default_rng(2)
    counts = r.integers(0, most + 1, b)
    mp = -(-most // page)
    s = state(3, b, h, page, mp, 0, free=b * h * mp, extra=b < 10)
    run(sa, s, spans_of(counts), int(counts.sum()) + 9, start=[0] * b)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("free", [0, 40, 4000])
def test_mixed(sa, seed, free):
    r = np.random.default_rng(seed + 10)
    b, h, page = int(r.integers(1, 40)), int(r.integers(1, 9)), int(r.choice([16, 32, 128]))
    mp = 40
    s = state(seed, b, h, page, mp, 20 * page, spare=6, free=free, extra=seed % 2 == 0)
    counts = r.integers(0, 10 * page, b) * (r.random(b) < 0.7)
    ended = (r.random(b) < 0.3).tolist()
    start = r.integers(0, 5000, b).tolist()
    spans = spans_of(counts, gap=int(r.integers(0, 3)))
    tokens = spans[-1][1] + 3
    ref = opg.grow(s["table"], s["lens"], s["owned"], s["free"], page, spans, counts, ended, start, tokens)
    short = (ref["granted"] != counts).any()
    run(sa, s, spans, tokens, counts.tolist(), ended, start, status=sa.SA_DEV_NO_PAGES if short else 0)


def test_new_state_apart_from_the_old(sa):
    # many CTAs, whose first one writes the new state at once: the old one stays as it is
    r = np.random.default_rng(3)
    s = state(4, 20, 3, 32, 60, 900, spare=5, free=300)
    counts = r.integers(0, 900, 20)
    spans, tokens = spans_of(counts), int(counts.sum())
    ended = (r.random(20) < 0.3).tolist()
    start = r.integers(0, 5000, 20).tolist()
    d, pool = to_gpu(sa, s)
    saved = {k: v.clone() for k, v in d.items() if v is not None}
    i32 = dict(dtype=torch.int32, device="cuda")
    out = {k: torch.full_like(d[k], 9) for k in ("lens", "owned", "free_count")}
    first, after, granted = torch.tensor(start, **i32), torch.zeros(20, **i32), torch.zeros(20, **i32)
    slots, pos = torch.zeros(3, tokens, dtype=torch.int64, device="cuda"), torch.zeros(tokens, **i32)
    cu = torch.tensor([0] + [e for _, e in spans], **i32)
    ref = opg.grow(s["table"], s["lens"], s["owned"], s["free"], 32, spans, None, ended, start, tokens)
    for _ in range(3):                                        # what it reads stays, so it can be done again
        pool.grow(slots, cu=cu, ended=torch.tensor(ended, device="cuda"), start=first, positions=pos, granted=granted,
                  lens_out=out["lens"], owned_out=out["owned"], free_count_out=out["free_count"], start_out=after)
        np.testing.assert_array_equal(slots.cpu(), ref["slots"])
        np.testing.assert_array_equal(pos.cpu(), ref["token_positions"])
        np.testing.assert_array_equal(out["lens"].cpu(), ref["lens"])
        np.testing.assert_array_equal(out["owned"].cpu(), ref["owned"])
        np.testing.assert_array_equal(after.cpu(), ref["start"])
        np.testing.assert_array_equal(granted.cpu(), ref["granted"])
        np.testing.assert_array_equal(d["table"].cpu(), ref["table"])
        assert int(out["free_count"]) == len(ref["free"])
        for k in ("lens", "owned", "free_count"):
            assert torch.equal(d[k], saved[k])
    assert first.tolist() == start


def test_a_pool_that_is_too_small(sa):
    # the second sequence wants more than there is; the third, which wants none, goes on; the fourth has to wait
    s = {"table": np.full((4, 1, 8), -1), "lens": np.array([[0], [0], [3], [0]]), "owned": np.array([[0], [0], [1], [0]]),
         "free": [4, 9, 2], "pages": 10, "page": 16}
    s["table"][2, 0, 0] = 7
    d, _, ref = run(sa, s, spans_of([20, 30, 5, 1]), 56, status=sa.SA_DEV_NO_PAGES)
    assert ref["granted"].tolist() == [20, 0, 5, 0] and d["table"][0, 0, :2].tolist() == [2, 9]


def test_steps_of_a_pool_give_back_all_pages(sa):
    b, h, page, mp, pages = 6, 3, 16, 12, 150
    r = np.random.default_rng(5)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.zeros(b, h, mp, **i32), torch.zeros(b, h, **i32)
    pool = sa.PagePool(table, lens, page, num_pages=pages)
    for step in range(60):
        counts = torch.tensor(r.integers(0, 30, b) * (r.random(b) < 0.5), **i32)
        counts = torch.minimum(counts, mp * page - lens.amax(1))
        ended = torch.tensor(r.random(b) < 0.1, device="cuda")
        slots = torch.zeros(h, b * 30, dtype=torch.int64, device="cuda")
        pool.grow(slots, counts=counts, ended=ended)
        if step % 7 == 3:                                     # rows cut, as an eviction does
            lens.copy_(torch.minimum(lens, torch.tensor(r.integers(0, 100, (b, h)), **i32)))
        owned = pool.owned.cpu().numpy()
        used = table.cpu().numpy()[np.arange(mp) < owned[..., None]].tolist()
        spare = pool.free_pages[:int(pool.free_count)].tolist()
        assert sorted(used + spare) == list(range(pages))
        got = slots[slots >= 0]
        assert got.unique().numel() == got.numel()
    lens.zero_()
    pool.grow(torch.zeros(h, 0, dtype=torch.int64, device="cuda"))
    assert int(pool.free_count) == pages and (pool.owned == 0).all()
    assert int(pool.dev_status) & ~sa.SA_DEV_NO_PAGES == 0


def test_bad_state_is_clamped_and_flagged(sa):
    def fresh():
        return to_gpu(sa, state(6, 4, 2, 16, 8, 100, free=40))

    slots = torch.zeros(2, 40, dtype=torch.int64, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 10, 20, 30, 40], **i32)

    def flagged(what, **kw):
        d, pool = fresh()
        what(d)
        pool.grow(slots, cu=kw.pop("cu", good), **kw)
        torch.cuda.synchronize()
        assert int(pool.dev_status.item()) & sa.SA_DEV_BAD_COUNT
        assert (pool.owned >= 0).all() and (pool.owned <= 8).all() and int(pool.free_count) <= pool.num_pages
        return d

    for name, value in (("lens", -3), ("lens", 200), ("lens", 2 ** 31 - 1), ("owned", -1), ("owned", 2 ** 30),
                        ("free_count", -5), ("free_count", 2 ** 31 - 1)):
        flagged(lambda d: d[name].view(-1)[0].fill_(value))
    for cu in ([0, 10, 5, 30, 40], [0, 10, 20, 30, 41], [-1, 10, 20, 30, 40], [2 ** 31 - 1, -2 ** 31, 0, 0, 0]):
        flagged(lambda d: None, cu=torch.tensor(cu, **i32))
        assert (slots == -1).all()                            # nobody's spans are known
    flagged(lambda d: None, counts=torch.tensor([11, -1, 5, 2 ** 31 - 1], **i32))
    # more tokens than the row's table has slots: none
    d, pool = to_gpu(sa, state(7, 1, 2, 16, 2, 0, free=40))
    pool.grow(slots, cu=torch.tensor([0, 33], **i32))
    assert int(pool.dev_status) == sa.SA_DEV_BAD_COUNT and (slots == -1).all() and (d["lens"] == 0).all()
    # page numbers out of range have no slots
    d, pool = fresh()
    d["free_pages"].fill_(10 ** 6)
    pool.grow(slots, cu=good)
    assert int(pool.dev_status) & sa.SA_DEV_BAD_INDEX
    assert ((slots >= -1) & (slots < pool.num_pages * 16)).all()


def test_streams_and_graphs(sa):
    s = state(8, 5, 2, 16, 30, 50, free=200, extra=True)
    d, pool = to_gpu(sa, s)
    slots = torch.zeros(2, 5, dtype=torch.int64, device="cuda")
    saved = {k: v.clone() for k, v in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.grow(slots)
    steps = []
    for _ in range(40):
        graph.replay()
        steps.append(slots.clone())
    end = {k: v.clone() for k, v in d.items()}
    for k, v in saved.items():
        d[k].copy_(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x in steps:
        pool.grow(slots, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(slots, x)
        side.wait_stream(torch.cuda.current_stream())
    assert all(torch.equal(d[k], end[k]) for k in end)
    assert int(pool.dev_status.item()) == 0


def test_steps_one_behind_the_other_on_used_shared_memory(sa):
    # other kernels leave their own values in shared memory, and launches overlap
    b, h, page = 64, 8, 16
    s = state(9, b, h, page, 501, 8000, free=b * h)
    d, pool = to_gpu(sa, s)
    att = sa.PackedAttention(8, 2, 64)
    q = torch.randn(300, 8, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    slots = torch.zeros(h, b, dtype=torch.int64, device="cuda")
    out = {k: torch.zeros_like(d[k]) for k in ("lens", "owned", "free_count")}
    ref = opg.grow(s["table"], s["lens"], s["owned"], s["free"], page, [(x, x + 1) for x in range(b)], tokens=b)
    for _ in range(40):
        att(q, q[:, :2], q[:, 2:4], cu)
        for _ in range(3):
            pool.grow(slots, lens_out=out["lens"], owned_out=out["owned"], free_count_out=out["free_count"])
    torch.cuda.synchronize()
    assert int(pool.dev_status.item()) == 0
    np.testing.assert_array_equal(slots.cpu().numpy(), ref["slots"])
    np.testing.assert_array_equal(out["lens"].cpu().numpy(), ref["lens"])
    np.testing.assert_array_equal(out["owned"].cpu().numpy(), ref["owned"])
    assert int(out["free_count"]) == len(ref["free"])
