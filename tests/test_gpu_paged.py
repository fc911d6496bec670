"""The paged cache operators on the GPU against the fp64 oracle."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa, torch


def _q(torch, seed, b, hq, d, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(b, hq, d, generator=g) * sharp).bfloat16()


def _attend(env, c, hq, out_dtype="bfloat16", weights=False, sharp=1.0, seed=5, **kw):
    from tests import _paged as P
    sa, torch = env
    b, hkv = c["lens"].shape
    d = c["k"].shape[2]
    q = _q(torch, seed, b, hq, d, sharp)
    dev, cache = P.to_gpu(c, sa)
    out = torch.full((b, hq, d), 7.0, dtype=getattr(torch, out_dtype), device="cuda")
    lse = torch.full((b, hq), 7.0, device="cuda")
    w = torch.full_like(dev["weights"], -3.0) if weights else None
    cache.attend(q.cuda(), out=out, lse=lse, weights_out=w, accumulate=weights, **kw)
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, out, lse, w)
    if weights:
        # slots behind a row's length stay as they were
        t = torch.arange(w.shape[-1])
        behind = t >= c["lens"][..., None]
        assert (w.cpu()[behind] == -3.0).all()
    return out, lse, w


EDGES = [0, 1, 15, 16, 17, 31, 33, 63, 64, 127, 128, 129, 255, 257, 700, 1025]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (7, 1, 128)])
def test_attend_lengths(env, page, hq, hkv, d):
    from tests import _paged as P
    c = P.random_cache(page + d, EDGES, hkv, d, page)
    _attend(env, c, hq, weights=True)
    _attend(env, c, hq, "float32")


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 9, 12, 16, 17, 20, 32, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_groups(env, G, d):
    from tests import _paged as P
    c = P.random_cache(G, [[300, 5], [0, 129], [64, 1000]], 2, d, 32)
    _attend(env, c, 2 * G, weights=True)
    _attend(env, c, 2 * G, "float32", weights=True)


@pytest.mark.parametrize("lens,hkv", [([20000], 1), ([9000, 1, 4097], 2), ([130] * 200, 4)])
def test_attend_splits_and_many_rows(env, lens, hkv):
    from tests import _paged as P
    c = P.random_cache(3, lens, hkv, 128, 64)
    _attend(env, c, 4 * hkv, weights=True)
    _attend(env, c, 4 * hkv, "float32")


@pytest.mark.parametrize("sharp", [0.0, 30.0])
def test_attend_flat_and_sharp_scores(env, sharp):
    # equal scores everywhere, and scores whose maximum grows far along the row
    from tests import _paged as P
    c = P.random_cache(8, [3000, 513], 2, 128, 16)
    c["k"][:] = (c["k"].float() * 1.0).bfloat16()
    _attend(env, c, 8, weights=True, sharp=sharp)
    _attend(env, c, 8, "float32", sharp=sharp)


def test_attend_growing_scores(env):
    # keys that score ever higher towards the row's end: the running maximum
    # moves in every piece
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(9, [2000], 1, 128, 32, junk=False)
    q = torch.ones(1, 4, 128).bfloat16()
    t = torch.arange(2000)
    p, x = c["table"][0, 0].long()[t // 32], t % 32
    c["k"][p, x] = (0.02 * (t // 8).float()[:, None].expand(-1, 128)).bfloat16()
    dev, cache = P.to_gpu(c, sa)
    out, lse = torch.empty(1, 4, 128, device="cuda"), torch.empty(1, 4, device="cuda")
    w = torch.zeros_like(dev["weights"])
    cache.attend(q.cuda(), out=out, lse=lse, weights_out=w)
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, out, lse, w)


def test_attend_strided_queries_and_interleaved_pools(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(10, [77, 300, 0], 2, 128, 32, interleaved=True)
    assert c["k"].stride(0) == 2 * 32 * 128
    dev, cache = P.to_gpu(c, sa)
    assert dev["k"].stride(0) == 2 * 32 * 128
    big = _q(torch, 1, 3, 30, 256)
    q = big[:, 3:27:3, 64:192]
    out = cache.attend(big.cuda()[:, 3:27:3, 64:192])
    assert out.dtype == torch.bfloat16 and out.shape == (3, 8, 128)
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, out, None)


def test_attend_adds_in_place_and_is_repeatable(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(11, [5000, 64, 1], 2, 128, 64)
    q = _q(torch, 2, 3, 8, 128)
    outs = []
    for _ in range(2):
        dev, cache = P.to_gpu(c, sa)
        o = cache.attend(q.cuda())
        outs.append((o, dev["weights"]))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    P.check_attend(c, q, outs[0][0], None, outs[0][1])
    t = torch.arange(c["weights"].shape[-1])
    behind = t >= c["lens"][..., None]
    assert torch.equal(outs[0][1].cpu()[behind], c["weights"][behind])
    # without accumulation the weights stay
    dev, cache = P.to_gpu(c, sa)
    o = cache.attend(q.cuda(), accumulate=False)
    assert torch.equal(o, outs[0][0]) and torch.equal(dev["weights"].cpu(), c["weights"])


def test_attend_propagates_nan_of_live_tokens_only_to_its_row(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(12, [100, 200], 1, 64, 16)
    t = 37
    c["v"][c["table"][0, 0, t // 16].long(), t % 16, 3] = float("nan")
    dev, cache = P.to_gpu(c, sa)
    o = cache.attend(_q(torch, 3, 2, 4, 64).cuda()).float().cpu()
    assert torch.isnan(o[0, :, 3]).all()
    o[0, :, 3] = 0
    assert torch.isfinite(o).all()


def test_attend_far_pages(env):
    # element offsets beyond 2^31 in both pools
    from tests import _paged as P
    sa, torch = env
    page, d, pages = 64, 128, (1 << 31) // (64 * 128) + 64
    k = torch.empty(pages, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(pages, page, d, dtype=torch.bfloat16, device="cuda")
    c = P.random_cache(13, [500], 1, d, page, spare=0)
    n = c["k"].shape[0]
    k[pages - n:], v[pages - n:] = c["k"].cuda(), c["v"].cuda()
    table = (c["table"] + (pages - n)).cuda()
    w, pos, lens = c["weights"].cuda(), c["positions"].cuda(), c["lens"].cuda()
    cache = sa.PagedCache(k, v, table, lens, weights=w, positions=pos)
    q = _q(torch, 4, 1, 4, d)
    o = cache.attend(q.cuda(), accumulate=False)
    P.check_attend(c, q, o, None)
    # append into the last slots, then evict across them
    kn = _q(torch, 5, 1, 5, d)[:, None].contiguous()
    vn = _q(torch, 6, 1, 5, d)[:, None].contiguous()
    cache.append(kn.cuda(), vn.cuda())
    from oracle import paged as op
    ref = op.append(P.f64(c["k"]), P.f64(c["v"]), c["table"].numpy(), c["lens"].numpy(), P.f64(kn),
                    P.f64(vn), [5], [500], P.f64(c["weights"]), c["positions"].numpy())
    cache.evict([300], 4, 16)
    ref = op.evict(ref[0], ref[1], c["table"].numpy(), *ref[2:], [300], 4, 16)
    assert int(cache.dev_status.item()) == 0
    used = P.slot_mask(c["table"], torch.as_tensor(ref[2]), page, n)
    assert np.array_equal(P.f64(k[pages - n:])[used], ref[0][used])
    assert np.array_equal(P.f64(v[pages - n:])[used], ref[1][used])
    assert lens.cpu().numpy().tolist() == ref[2].tolist()
    assert np.array_equal(P.f64(w)[0, 0, :300], ref[3][0, 0, :300])


@pytest.mark.parametrize("Bt,hkv,d,page,T", [(3, 2, 128, 16, 1), (70, 8, 128, 32, 1),
                                             (2, 2, 64, 64, 1), (4, 2, 128, 32, 37),
                                             (3, 1, 64, 256, 300), (1, 4, 128, 128, 1000)])
@pytest.mark.parametrize("inplace", [True, False])
def test_append(env, Bt, hkv, d, page, T, inplace):
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    r = np.random.default_rng(Bt * T)
    lens = r.integers(0, 400, Bt)
    counts = r.integers(0, T + 1, Bt).astype(np.int32)
    counts[0] = T
    start = r.integers(0, 1000, Bt).astype(np.int32)
    c = P.random_cache(T, lens + T, hkv, d, page, junk=False)     # pages for all of them
    c["lens"] = torch.as_tensor(lens, dtype=torch.int32)[:, None].expand(-1, hkv).contiguous()
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn(Bt, T, 3 * hkv, d, generator=g).bfloat16()  # a fused projection's output
    kn, vn = qkv[:, :, hkv:2 * hkv].transpose(1, 2), qkv[:, :, 2 * hkv:].transpose(1, 2)
    dev, cache = P.to_gpu(c, sa)
    gq = qkv.cuda()
    lens_out = None if inplace else torch.full_like(dev["lens"], -1)
    cache.append(gq[:, :, hkv:2 * hkv].transpose(1, 2), gq[:, :, 2 * hkv:].transpose(1, 2),
                 counts=torch.as_tensor(counts).cuda(), start=torch.as_tensor(start).cuda(),
                 lens_out=lens_out)
    assert int(cache.dev_status.item()) == 0
    k, v, l, w, p = op.append(P.f64(c["k"]), P.f64(c["v"]), c["table"].numpy(), c["lens"].numpy(),
                              P.f64(kn), P.f64(vn), counts, start, P.f64(c["weights"]),
                              c["positions"].numpy())
    assert np.array_equal(P.f64(dev["k"]), k) and np.array_equal(P.f64(dev["v"]), v)
    assert np.array_equal((dev["lens"] if inplace else lens_out).cpu().numpy(), l)
    if not inplace:
        assert torch.equal(dev["lens"].cpu(), c["lens"])
    assert np.array_equal(P.f64(dev["weights"]), w)
    assert np.array_equal(dev["positions"].cpu().numpy(), p)


def test_append_defaults_and_overflow(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(21, [10, 32], 1, 64, 16, max_pages=2, junk=False)
    c["table"][0, 0, 1] = c["table"].max() + 1
    c["table"][0, 0, 1] = [x for x in range(c["k"].shape[0]) if x not in c["table"].flatten().tolist()][0]
    dev, cache = P.to_gpu(c, sa)
    kn = torch.randn(2, 1, 4, 64).bfloat16()
    cache.append(kn.cuda(), kn.cuda())           # row 1 is full: its tokens are dropped
    assert int(cache.dev_status.item()) == sa.SA_DEV_BAD_COUNT
    assert dev["lens"].flatten().tolist() == [14, 32]
    k = dev["k"].cpu()
    page, x = c["table"][0, 0, 0].item(), torch.arange(10, 14)
    assert torch.equal(k[page, x], kn[0, 0])
    k[page, x] = c["k"][page, x]
    assert torch.equal(k, c["k"])
    assert dev["positions"][0, 0, 10:14].tolist() == [10, 11, 12, 13]
    assert (dev["weights"][0, 0, 10:14] == 0).all()


def test_out_of_range_pages_and_lengths_are_flagged_not_used(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(22, [100, 60], 1, 128, 32, junk=False)
    c["table"][0, 0, 1] = c["k"].shape[0]
    c["table"][1, 0, 0] = -5
    before = c["k"].clone()
    dev, cache = P.to_gpu(c, sa)
    out = cache.attend(_q(torch, 7, 2, 4, 128).cuda())
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == sa.SA_DEV_BAD_INDEX
    assert torch.isfinite(out.float()).all()
    dev["table"][0, 0, 3] = 1 << 30              # the page that the next tokens go to
    cache.dev_status.zero_()
    kn = torch.randn(2, 1, 2, 128).bfloat16().cuda()
    cache.append(kn, kn, counts=torch.tensor([2, 0], dtype=torch.int32).cuda())
    assert int(cache.dev_status.item()) == sa.SA_DEV_BAD_INDEX
    assert torch.equal(dev["k"].cpu(), before)
    assert dev["lens"].flatten().tolist() == [102, 60]
    # lengths out of range are clamped
    for bad, clamped in ((-7, 0), (1 << 30, cache.slots)):
        dev, cache = P.to_gpu(P.random_cache(22, [100, 60], 1, 128, 32, junk=False), sa)
        dev["table"].clamp_(min=0)
        dev["lens"][0, 0] = bad
        cache.attend(_q(torch, 7, 2, 4, 128).cuda())
        assert int(cache.dev_status.item()) == sa.SA_DEV_BAD_COUNT
        cache.dev_status.zero_()
        cache.evict([40], 2, 2)
        assert int(cache.dev_status.item()) == sa.SA_DEV_BAD_COUNT
        assert dev["lens"].flatten().tolist() == [min(clamped, 40), 40]


def _evict_case(torch, c, kind, seed):
    g = torch.Generator().manual_seed(seed)
    w = c["weights"]
    if kind == "random":
        w.copy_(torch.exp(2 * torch.randn(w.shape, generator=g)))
    elif kind == "ties":
        w.copy_(torch.randint(0, 3, w.shape, generator=g).float())
    elif kind == "zeros":
        w.zero_()
        w[..., ::2] = -0.0
    elif kind == "odd":
        vals = torch.tensor([float("nan"), float("inf"), -float("inf"), -1.0, 0.0, -0.0, 1e-40, 2.0])
        w.copy_(vals[torch.randint(0, 8, w.shape, generator=g)])
    pos = torch.argsort(torch.rand(c["positions"].shape, generator=g), -1).int() * 2
    c["positions"].copy_(pos)


@pytest.mark.parametrize("kind", ["random", "ties", "zeros", "odd"])
@pytest.mark.parametrize("lens,keep,sinks,recent,d,page", [
    ([[300, 40], [0, 1], [64, 1000]], [64, 50], 4, 16, 128, 32),
    ([[300, 40], [1, 2], [512, 513]], [0, 1], 0, 0, 64, 16),
    ([[5000, 4100], [2049, 33]], [2048, 700], 0, 100, 128, 64),
    ([[700, 700]], [700, 699], 10, 0, 64, 256),
    ([[20000, 9999]], [128, 9000], 4, 64, 64, 128),
])
def test_evict(env, kind, lens, keep, sinks, recent, d, page):
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(31, lens, 2, d, page, junk=False)
    _evict_case(torch, c, kind, 5)
    ref = op.evict(P.f64(c["k"]), P.f64(c["v"]), c["table"].numpy(), c["lens"].numpy(),
                   c["weights"].numpy(), c["positions"].numpy(), keep, sinks, recent)
    t = torch.arange(c["weights"].shape[-1])
    live = (t < torch.as_tensor(ref[2])[..., None]).numpy()
    for inplace in (True, False):
        dev, cache = P.to_gpu(c, sa)
        outs = {}
        if not inplace:
            outs = {"lens_out": torch.full_like(dev["lens"], -9),
                    "weights_out": torch.full_like(dev["weights"], -9.0),
                    "positions_out": torch.full_like(dev["positions"], -9)}
        cache.evict(keep, sinks, recent, **outs)
        assert int(cache.dev_status.item()) == 0
        assert np.array_equal(P.f64(dev["k"]), ref[0]) and np.array_equal(P.f64(dev["v"]), ref[1])
        got = [dev["lens"], dev["weights"], dev["positions"]] if inplace else list(outs.values())
        assert np.array_equal(got[0].cpu().numpy(), ref[2])
        assert np.array_equal(got[1].cpu().numpy()[live], ref[3][live], equal_nan=True)
        assert np.array_equal(got[2].cpu().numpy()[live], ref[4][live])
        if inplace:
            assert np.array_equal(got[1].cpu().numpy()[~live], c["weights"].numpy()[~live], equal_nan=True)
            assert np.array_equal(got[2].cpu().numpy()[~live], c["positions"].numpy()[~live])
        else:
            assert (got[1].cpu().numpy()[~live] == -9).all() and (got[2].cpu().numpy()[~live] == -9).all()
            assert torch.equal(dev["lens"].cpu(), c["lens"])
            assert np.array_equal(P.f64(dev["weights"]), P.f64(c["weights"]), equal_nan=True)


def test_evict_without_positions(env):
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(32, [500, 100], 1, 128, 32, junk=False)
    dev, _ = P.to_gpu(c, sa)
    cache = sa.PagedCache(dev["k"], dev["v"], dev["table"], dev["lens"], weights=dev["weights"])
    cache.evict([120], 8, 32)
    ref = op.evict(P.f64(c["k"]), P.f64(c["v"]), c["table"].numpy(), c["lens"].numpy(),
                   c["weights"].numpy(), c["positions"].numpy(), [120], 8, 32)
    assert int(cache.dev_status.item()) == 0
    assert np.array_equal(P.f64(dev["k"]), ref[0]) and np.array_equal(dev["lens"].cpu().numpy(), ref[2])
    assert np.array_equal(dev["weights"].cpu().numpy(), ref[3])


def test_decode_loop_with_evictions(env):
    # append, attend with weights and evict in turn, as a serving loop runs
    # them; the oracle follows on the GPU's own weights, so that a rounding of
    # a weight cannot turn into another eviction
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    Bt, hkv, hq, d, page, keep = 2, 2, 8, 128, 16, [48, 80]
    c = P.random_cache(41, [[60, 90], [33, 100]], hkv, d, page, max_pages=8, spare=20, junk=False)
    free = [x for x in range(c["k"].shape[0]) if x not in c["table"].flatten().tolist()]
    for b in range(Bt):
        for g in range(hkv):
            for i in range(8):
                if c["table"][b, g, i] < 0 and i < 7 and free:
                    c["table"][b, g, i] = free.pop()
    dev, cache = P.to_gpu(c, sa, num_q_heads=hq)
    gen = torch.Generator().manual_seed(3)
    for step in range(24):
        kn = torch.randn(Bt, hkv, 1, d, generator=gen).bfloat16()
        vn = torch.randn(Bt, hkv, 1, d, generator=gen).bfloat16()
        q = torch.randn(Bt, hq, d, generator=gen).bfloat16()
        start = torch.full((Bt,), 200 + step, dtype=torch.int32)
        state = {n: dev[n].cpu() for n in ("k", "v", "table", "lens", "weights", "positions")}
        cache.append(kn.cuda(), vn.cuda(), start=start.cuda())
        ref = op.append(P.f64(state["k"]), P.f64(state["v"]), state["table"].numpy(),
                        state["lens"].numpy(), P.f64(kn), P.f64(vn), [1] * Bt, start.numpy(),
                        P.f64(state["weights"]), state["positions"].numpy())
        assert np.array_equal(P.f64(dev["k"]), ref[0]) and np.array_equal(dev["lens"].cpu().numpy(), ref[2])
        after = {n: dev[n].cpu() for n in ("k", "v", "table", "lens", "weights", "positions")}
        lse = torch.empty(Bt, hq, device="cuda")
        o = cache.attend(q.cuda(), lse=lse)
        P.check_attend({**after, "page": page}, q, o, lse, dev["weights"], after["weights"])
        if step % 8 == 7:
            state = {n: dev[n].cpu() for n in ("k", "v", "table", "lens", "weights", "positions")}
            cache.evict(keep, 4, 8)
            ref = op.evict(P.f64(state["k"]), P.f64(state["v"]), state["table"].numpy(),
                           state["lens"].numpy(), state["weights"].numpy(),
                           state["positions"].numpy(), keep, 4, 8)
            assert np.array_equal(P.f64(dev["k"]), ref[0]) and np.array_equal(P.f64(dev["v"]), ref[1])
            assert np.array_equal(dev["lens"].cpu().numpy(), ref[2])
            for b in range(Bt):
                for g in range(hkv):
                    m = int(ref[2][b, g])
                    assert np.array_equal(dev["weights"].cpu().numpy()[b, g, :m], ref[3][b, g, :m])
                    assert np.array_equal(dev["positions"].cpu().numpy()[b, g, :m], ref[4][b, g, :m])
    assert int(cache.dev_status.item()) == 0


def test_captured_steps_follow_the_state(env):
    # append + attend captured once; each replay reads the lengths of its time
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(42, [100, 250], 2, 64, 16, max_pages=20, spare=60, junk=False)
    free = [x for x in range(c["k"].shape[0]) if x not in c["table"].flatten().tolist()]
    c["table"][c["table"] < 0] = torch.tensor(free[:int((c["table"] < 0).sum())], dtype=torch.int32)
    dev, cache = P.to_gpu(c, sa, num_q_heads=8)
    kv = torch.zeros(2, 2, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(2, 8, 64, device="cuda"), torch.empty(2, 8, device="cuda")
    lens0 = dev["lens"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(kv[0], kv[1])
        cache.attend(q, out=out, lse=lse)
    assert torch.equal(dev["lens"], lens0)
    for step in range(5):
        kv.copy_(torch.randn(kv.shape, device="cuda"))
        q.copy_(torch.randn(q.shape, device="cuda"))
        before = dev["weights"].cpu().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dev["lens"], lens0 + step + 1)
        now = {n: dev[n].cpu() for n in ("k", "v", "table", "lens", "weights")}
        for b in range(2):
            for h in range(2):
                before[b, h, int(now["lens"][b, h]) - 1] = 0       # the appended token's weight
        P.check_attend({**now, "page": 16}, q.cpu(), out, lse, dev["weights"], before)
    assert int(cache.dev_status.item()) == 0


def test_calls_on_a_given_stream(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(43, [900, 30], 2, 128, 32)
    dev, cache = P.to_gpu(c, sa)
    q = _q(torch, 9, 2, 8, 128)
    gq = q.cuda()
    ref = cache.attend(gq, accumulate=False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = cache.attend(gq, accumulate=False, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        b = cache.attend(gq, accumulate=False)
    side.synchronize()
    e = cache.attend(gq, accumulate=False, stream=side.cuda_stream)
    side.synchronize()
    for x in (a, b, e):
        assert torch.equal(x, ref)


def test_python_class_refusals(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(44, [20], 2, 64, 16)
    dev, cache = P.to_gpu(c, sa)
    q = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (q.float(), q[:, :7], q[0], q[:, :, :32], q.cpu(), q.expand(2, 8, 64)):
        with pytest.raises((ValueError, TypeError, sa.SparseAttnError)):
            cache.attend(bad)
    with pytest.raises((ValueError, sa.SparseAttnError)):
        cache.attend(q[:, :1].expand(1, 8, 64))          # heads on top of one another
    with pytest.raises(TypeError):
        cache.attend(q, out=torch.empty(1, 8, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        cache.attend(q, lse=torch.empty(8, device="cuda"))
    with pytest.raises(ValueError):
        cache.attend(q, accumulate=False, weights_out=dev["weights"])
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    for bad in ((k.float(), k), (k, k[:, :, :2]), (k[:, :1], k[:, :1]), (k[:, :, :0], k[:, :, :0]), (k.cpu(), k)):
        with pytest.raises((ValueError, TypeError)):
            cache.append(*bad)
    with pytest.raises(ValueError):
        cache.append(k, k, counts=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        cache.evict([10])
    with pytest.raises(sa.SparseAttnError):
        cache.evict([10, 3], 2, 2)
    for bad in (([2**32 + 50, 50], 0, 0), ([50, -1], 0, 0), ([50, 50], -1, 0), ([50, 50], 0, 2**32)):
        with pytest.raises(ValueError):
            cache.evict(*bad)
    plain = sa.PagedCache(dev["k"], dev["v"], dev["table"], dev["lens"])
    with pytest.raises(ValueError):
        plain.evict([10, 10])
    with pytest.raises(ValueError):
        plain.attend(q, accumulate=True)
    assert int(cache.dev_status.item()) == 0
    with pytest.raises(ValueError):
        sa.PagedCache(dev["k"].transpose(1, 2), dev["v"].transpose(1, 2), dev["table"], dev["lens"])
    with pytest.raises(ValueError):
        sa.PagedCache(dev["k"], dev["v"], dev["table"], dev["lens"], weights=dev["weights"][..., :-1].contiguous())


def test_attend_wait_limit_ends_the_launch(env):
    # every copy takes longer than 1 ns: the waits give up, the launch ends and
    # the next one, with the default limit, is right again
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(45, [3000, 200], 2, 128, 32)
    dev, cache = P.to_gpu(c, sa)
    q = _q(torch, 9, 2, 8, 128)
    gq = q.cuda()
    sa.sparse_attn_set_wait_limit(1)
    try:
        cache.attend(gq, accumulate=False)
        torch.cuda.synchronize()
    finally:
        sa.sparse_attn_set_wait_limit(0)
    assert int(cache.dev_status.item()) & sa.SA_DEV_TIMEOUT
    cache.dev_status.zero_()
    out, lse = torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, device="cuda")
    cache.attend(gq, out=out, lse=lse, accumulate=False)
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, out, lse)


def test_paged_decode_layer_follows_the_oracle(env):
    # prompts of two lengths from the prefill layout, steps with evictions to
    # per-head budgets, a sequence released and another admitted in its place
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    Bt, hkv, hq, d, page, keep = 3, 2, 8, 128, 16, [40, 90]
    layer = PagedDecodeLayer(Bt, hq, hkv, d, page, num_pages=80, max_tokens=200, keep=keep,
                             slack=8, sinks=4, recent=8)
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen).bfloat16()

    def state():
        return {"k": layer.k_pages.cpu(), "v": layer.v_pages.cpu(), "table": layer.table.cpu(),
                "lens": layer.lens.cpu(), "weights": layer.weights.cpu(),
                "positions": layer.positions.cpu(), "page": page}

    def rows_of(s, b, g):
        n = int(s["lens"][b, g])
        p, x = op.slot_rows(s["table"][b, g].numpy(), np.arange(n), page)
        return s["k"][p, x], s["positions"][b, g, :n]

    kept = {}                        # (sequence, position) -> key rows, of everything appended

    def admit(b, tokens):
        k, v = rnd(hkv, tokens, d), rnd(hkv, tokens, d)
        for t in range(tokens):
            kept[b, t] = k[:, t]
        layer.admit(b, k.cuda(), v.cuda(), queries=rnd(3, hq, d).cuda())
        return tokens

    pos = {0: admit(0, 30), 1: admit(1, 150)}
    assert layer.lens.tolist() == [[30, 30], [40, 90], [0, 0]]
    for step in range(40):
        if step == 15:
            layer.release(0)
            del pos[0]
        if step == 17:
            pos[0] = admit(0, 70)
        if step == 20:
            pos[2] = admit(2, 1)
        q, k, v = rnd(Bt, hq, d), rnd(Bt, hkv, d), rnd(Bt, hkv, d)
        before = state()
        lse = torch.empty(Bt, hq, device="cuda")
        out = layer.step(q.cuda(), k.cuda(), v.cuda(), lse=lse).clone()
        for b in pos:
            kept[b, pos[b]] = k[b]
            pos[b] += 1
        assert int(layer.cache.dev_status.item()) == 0
        now = state()
        assert now["lens"].tolist() == layer.book.lens
        # the attention saw the old tokens and the new one (the device table is
        # only added to: after an eviction it still names the pages read)
        counts = [int(b in pos) for b in range(Bt)]
        ref = op.append(P.f64(before["k"]), P.f64(before["v"]), now["table"].numpy(),
                        before["lens"].numpy(), P.f64(k[:, :, None]), P.f64(v[:, :, None]), counts,
                        [pos.get(b, 1) - 1 for b in range(Bt)], P.f64(before["weights"]),
                        before["positions"].numpy())
        c = {"k": torch.as_tensor(ref[0]), "v": torch.as_tensor(ref[1]), "table": now["table"],
             "lens": torch.as_tensor(ref[2]), "weights": torch.as_tensor(ref[3]), "page": page}
        P.check_attend(c, q, out, lse)
        # what is left are tokens that were appended, each with its own key,
        # the first and the last positions among them
        for b in pos:
            for g in range(hkv):
                rows, p = rows_of(now, b, g)
                assert len(set(p.tolist())) == len(p)
                for row, x in zip(rows, p.tolist()):
                    assert torch.equal(row, kept[b, x][g])
                for x in list(range(min(4, pos[b]))) + list(range(max(0, pos[b] - 8), pos[b])):
                    assert x in p.tolist()
        for b in range(Bt):
            if b not in pos:
                assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()


def test_paged_decode_layer_after_the_prefill_layer(env):
    # the prefill layer's keys and values, a plan's budgets: one layer of a
    # served prompt, with and without room for everything
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer, PrefillLayer, kv_budgets
    from tests import _paged as P
    from tests._parity import to_dev
    sa, torch = env
    from workloads import generate, scaled, workload
    w = scaled(workload(1), 1024)
    x = generate.prefill_inputs(w)
    t = {n: to_dev(x[n]) for n in "qkv"}
    shape = sa.Shape.prefill(w.seq_len, w.block, w.num_q_heads, w.num_kv_heads, w.head_dim)
    pre = PrefillLayer(shape, 6, demand=[3, 5, 4, 9, 2, 2, 8, 4], num_workers=8)
    pre(t["q"], t["k"], t["v"])
    keep = kv_budgets(pre.plan, w.block)
    budgets = pre.plan.get()["budgets"]
    assert keep == [int(budgets[:4].max()) * 64, int(budgets[4:].max()) * 64]
    q = _q(torch, 3, 1, 8, 64)
    kn, vn = _q(torch, 4, 1, 2, 64), _q(torch, 5, 1, 2, 64)
    for budget in (None, keep):
        layer = PagedDecodeLayer(1, 8, 2, 64, 64, num_pages=40, max_tokens=1100, keep=budget,
                                 slack=0)
        layer.admit(0, t["k"], t["v"], queries=t["q"].transpose(0, 1)[-4:])
        lens = [1024, 1024] if budget is None else [min(1024, n) for n in keep]
        assert layer.lens.tolist() == [lens]
        lse = torch.empty(1, 8, device="cuda")
        out = layer.step(q.cuda(), kn.cuda(), vn.cuda(), lse=lse).clone()
        assert int(layer.cache.dev_status.item()) == 0
        if budget is None:
            k = torch.cat([t["k"].cpu(), kn[0][:, None]], 1)
            v = torch.cat([t["v"].cpu(), vn[0][:, None]], 1)
            c = {"k": k.view(2, 1025, 64), "v": v.view(2, 1025, 64),
                 "table": torch.tensor([[[0], [1]]], dtype=torch.int32),
                 "lens": torch.tensor([[1025, 1025]], dtype=torch.int32), "page": 1025,
                 "weights": None}
            P.check_attend(c, q, out, lse)
        else:
            assert layer.lens.tolist() == [lens]           # cut back to the budgets
            assert len(layer.book.free) == 40 - sum(-(-n // 64) for n in lens)


def test_paged_decode_layer_refusals(env):
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    sa, torch = env
    with pytest.raises(ValueError):
        PagedDecodeLayer(1, 8, 2, 64, 16, 10, 100, keep=[10, 30])
    with pytest.raises(sa.SparseAttnError):
        PagedDecodeLayer(1, 8, 2, 64, 24, 10, 100)
    layer = PagedDecodeLayer(2, 8, 2, 64, 16, 10, 100)
    k = torch.zeros(2, 70, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        layer.admit(0, k.float(), k)
    assert len(layer.book.free) == 10
    layer.admit(0, k, k)
    with pytest.raises(ValueError):
        layer.admit(0, k, k)
    with pytest.raises(MemoryError):
        layer.admit(1, k, k)                               # ten pages are all there are
    assert layer.active == [True, False] and layer.lens.tolist() == [[70, 70], [0, 0]]
    layer.release(0)
    layer.admit(1, k, k)
    assert layer.lens.tolist() == [[0, 0], [70, 70]]


def test_attend_sequences_that_share_pages(env):
    # a common prefix: the same page numbers in two rows' tables, and twice in
    # one row's
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(51, [200, 200, 200], 1, 128, 32)
    c["table"][1, 0, :4] = c["table"][0, 0, :4]
    c["table"][2, 0, 1] = c["table"][2, 0, 0]
    _attend(env, c, 8, weights=True)


def test_two_caches_at_the_same_time_on_two_streams(env):
    from tests import _paged as P
    sa, torch = env
    cases = [P.random_cache(52, [3000, 700], 2, 128, 16), P.random_cache(53, [900, 4100, 5], 2, 64, 64)]
    qs = [_q(torch, 20 + i, c["lens"].shape[0], 8, c["k"].shape[2]) for i, c in enumerate(cases)]
    made = [P.to_gpu(c, sa) for c in cases]
    gq = [q.cuda() for q in qs]
    outs = [torch.empty(q.shape, device="cuda") for q in qs]
    ws = [torch.zeros_like(dev["weights"]) for dev, _ in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (dev, cache), q, o, w, st in zip(made, gq, outs, ws, streams):
            cache.attend(q, out=o, weights_out=w, stream=st)
    torch.cuda.synchronize()
    for c, (dev, cache), q, o, w in zip(cases, made, qs, outs, ws):
        assert int(cache.dev_status.item()) == 0
        P.check_attend(c, q, o, None, w)


def test_two_graphs_that_share_a_cache(env):
    # each keeps nothing in the workspace that the other's replay could spoil
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(54, [2500, 100], 2, 128, 32)
    dev, cache = P.to_gpu(c, sa, num_q_heads=16)
    qs = [_q(torch, 30, 2, 8, 128), _q(torch, 31, 2, 16, 128)]
    gq = [q.cuda() for q in qs]
    outs = [torch.empty(q.shape, device="cuda") for q in qs]
    ws = [torch.zeros_like(dev["weights"]) for _ in qs]
    for q, o, w in zip(gq, outs, ws):
        cache.attend(q, out=o, weights_out=w)
    graphs = []
    for q, o, w in zip(gq, outs, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attend(q, out=o, weights_out=w)
        graphs.append(g)
    for o in outs:
        o.fill_(9)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == 0
    for q, o, w in zip(qs, outs, ws):
        P.check_attend(c, q, o, None, w)


def test_evict_captured_and_replayed(env):
    # a captured eviction works on the lengths and weights of its replay
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(55, [[300, 80], [120, 511]], 2, 64, 32, junk=False)
    dev, cache = P.to_gpu(c, sa)
    keep = [100, 64]
    graph = torch.cuda.CUDAGraph()
    cache.evict([2000, 2000])                      # keeps everything
    with torch.cuda.graph(graph):
        cache.evict(keep, 4, 8)
    assert torch.equal(dev["lens"].cpu(), c["lens"])
    for step in range(2):
        if step:
            dev["lens"].copy_(torch.tensor([[90, 64], [101, 65]], dtype=torch.int32))
            dev["weights"].copy_(torch.rand(dev["weights"].shape, device="cuda"))
        s = {n: dev[n].cpu() for n in ("k", "v", "lens", "weights", "positions")}
        graph.replay()
        torch.cuda.synchronize()
        ref = op.evict(P.f64(s["k"]), P.f64(s["v"]), c["table"].numpy(), s["lens"].numpy(),
                       s["weights"].numpy(), s["positions"].numpy(), keep, 4, 8)
        assert np.array_equal(P.f64(dev["k"]), ref[0]) and np.array_equal(P.f64(dev["v"]), ref[1])
        assert np.array_equal(dev["lens"].cpu().numpy(), ref[2])
        assert np.array_equal(dev["weights"].cpu().numpy(), ref[3])
        assert np.array_equal(dev["positions"].cpu().numpy(), ref[4])
    assert int(cache.dev_status.item()) == 0


@pytest.mark.parametrize("lens,hkv", [([8192, 8191], 2), ([8193, 12000], 1), ([70000], 1),
                                      ([262144], 1)])
def test_evict_row_lengths_at_the_kernels_borders(env, lens, hkv):
    # one CTA up to 8192 slots, clusters of 2 to 8 above; few rows with much to
    # move take a second launch.  Compared through the positions, which name
    # the tokens.
    from oracle import paged as op
    sa, torch = env
    b, page, d = len(lens), 32, 64
    cap = -(-max(lens) // page) * page
    g = torch.Generator().manual_seed(cap)
    pages = b * hkv * cap // page
    k = torch.randn(pages, page, d, device="cuda").bfloat16()
    v = torch.randn(pages, page, d, device="cuda").bfloat16()
    table = torch.randperm(pages, generator=g).int().view(b, hkv, -1)
    w = torch.randint(0, 5000, (b, hkv, cap), generator=g).float()      # many ties
    pos = torch.arange(cap, dtype=torch.int32).expand(b, hkv, cap).contiguous()
    n = torch.tensor(lens, dtype=torch.int32)[:, None].expand(b, hkv).contiguous()
    dev = [t.cuda() for t in (table, n, w, pos)]
    cache = sa.PagedCache(k, v, dev[0], dev[1], weights=dev[2], positions=dev[3])
    k0, v0 = k.clone(), v.clone()
    for keep in (cap * 2 // 3, 777):
        before = [x.cpu() for x in (dev[1], dev[2], dev[3])]
        cache.evict([keep] * hkv, 4, 32)
        torch.cuda.synchronize()
        assert int(cache.dev_status.item()) == 0
        for x in range(b):
            for y in range(hkv):
                m0 = int(before[0][x, y])
                kept = op.kept_slots(before[1][x, y, :m0].numpy(), before[2][x, y, :m0].numpy(),
                                     min(m0, keep), 4, 32)
                m = len(kept)
                slots = list(range(m))
                have = set(kept)
                for hole, src in zip([t for t in range(m) if t not in have],
                                     [t for t in kept if t >= m]):
                    slots[hole] = src
                assert int(dev[1][x, y]) == m
                assert torch.equal(dev[2][x, y, :m].cpu(), before[1][x, y][slots])
                assert torch.equal(dev[3][x, y, :m].cpu(), before[2][x, y][slots])
                # the rows of the pools follow the positions (slots at first)
                at = dev[0][x, y].long()
                now = torch.arange(m, device="cuda")
                was = dev[3][x, y, :m].long()
                assert torch.equal(k[at[now // page], now % page], k0[at[was // page], was % page])
                assert torch.equal(v[at[now // page], now % page], v0[at[was // page], was % page])


def test_evict_equal_positions_all_forced(env):
    # more forced tokens than the budget: the lower slots stay
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(56, [200], 1, 64, 16, junk=False)
    c["positions"].fill_(3)
    dev, cache = P.to_gpu(c, sa)
    k0 = dev["k"].clone()
    cache.evict([50], 0, 4)
    assert int(dev["lens"]) == 50 and torch.equal(dev["k"], k0)
    assert torch.equal(dev["weights"].cpu(), c["weights"])


def test_a_captured_call_keeps_its_workspace(env):
    # the workspace grows after a capture; the graph's replays still own theirs
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(57, [3000, 300], 2, 128, 32)
    dev, cache = P.to_gpu(c, sa, with_weights=False, num_q_heads=8)
    q = _q(torch, 40, 2, 8, 128)
    gq, out = q.cuda(), torch.zeros(2, 8, 128, device="cuda")
    cache.attend(gq, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(gq, out=out)
    before = cache._ws_bytes
    cache.attend(_q(torch, 41, 2, 64, 128).cuda())
    assert cache._ws_bytes > before
    torch.cuda.synchronize()
    junk = [torch.zeros(before // 4, dtype=torch.int32, device="cuda") for _ in range(4)]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(int(j.count_nonzero()) == 0 for j in junk)
    P.check_attend(c, q, out, None)


def test_another_streams_call_takes_no_memory_the_current_one_still_uses(env):
    # the current stream has freed a block and is still to write it
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(58, [700, 90], 2, 128, 32)
    dev, cache = P.to_gpu(c, sa, with_weights=False)
    q = _q(torch, 42, 2, 8, 128)
    gq = q.cuda()
    need = sa.sparse_attn_paged_attend_workspace_size(cache.desc, 8, False)
    torch.cuda.synchronize()
    for other in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        torch.cuda._sleep(20_000_000)
        busy = [torch.full((need,), 7, dtype=torch.uint8, device="cuda"),
                torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")]
        spans = [(x.data_ptr(), x.data_ptr() + x.nbytes) for x in busy]
        del busy
        out = cache.attend(gq, stream=other)
        for x in (out, cache._ws):
            assert all(x.data_ptr() + x.nbytes <= a or b <= x.data_ptr() for a, b in spans)
        torch.cuda.synchronize()
        P.check_attend(c, q, out, None)


def test_paged_decode_layer_refused_calls_change_nothing(env):
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    from tests import _paged as P
    sa, torch = env
    layer = PagedDecodeLayer(2, 8, 2, 64, 16, 20, 200, keep=[40, 40], slack=80)
    gen = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=gen).bfloat16()
    k, v = rnd(2, 32, 64), rnd(2, 32, 64)
    with pytest.raises(ValueError):                        # queries of the wrong width
        layer.admit(0, k.cuda(), v.cuda(), queries=rnd(1, 8, 128).cuda())
    assert not layer.active[0] and len(layer.book.free) == 20 and not layer.lens.any()
    layer.admit(0, k.cuda(), v.cuda())
    q, k1, v1 = rnd(2, 8, 64), rnd(2, 2, 64), rnd(2, 2, 64)
    gq, gk, gv = q.cuda(), k1.cuda(), v1.cuda()
    for bad in ((gq, gk.float(), gv), (gq[:1], gk, gv), (gq.float(), gk, gv)):
        with pytest.raises((TypeError, ValueError)):       # the new token opens a page
            layer.step(*bad)
        assert layer.lens.tolist() == layer.book.lens == [[32, 32], [0, 0]]
        assert len(layer.book.free) == 16 and layer.start.tolist() == [32, 0]
    lse = torch.empty(2, 8, device="cuda")
    out = layer.step(gq, gk, gv, lse=lse)
    assert layer.lens.tolist() == layer.book.lens == [[33, 33], [0, 0]]
    c = {"k": torch.zeros(3, 33, 64).bfloat16(), "v": torch.zeros(3, 33, 64).bfloat16(),
         "table": torch.tensor([[[0], [1]], [[2], [2]]], dtype=torch.int32),
         "lens": torch.tensor([[33, 33], [0, 0]], dtype=torch.int32), "page": 33, "weights": None}
    c["k"][:2] = torch.cat([k, k1[0][:, None]], 1)
    c["v"][:2] = torch.cat([v, v1[0][:, None]], 1)
    P.check_attend(c, q, out, lse)


def test_handle_zero_is_the_default_stream(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(59, [300], 2, 64, 16)
    dev, cache = P.to_gpu(c, sa, with_weights=False, num_q_heads=4)
    q = _q(torch, 43, 1, 4, 64)
    late = q.cuda()
    gq = torch.zeros_like(late)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    gq.copy_(late)                                 # the default stream's, still to come
    with torch.cuda.stream(torch.cuda.Stream()):
        out = cache.attend(gq, stream=0)
    torch.cuda.synchronize()
    P.check_attend(c, q, out, None)


def test_paged_decode_layer_gone_while_another_stream_works(env):
    # the layer is dropped with its step still queued on a side stream: its
    # memory is not handed to the first stream before that step has run
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    sa, torch = env
    layer = PagedDecodeLayer(1, 8, 2, 64, 16, 20, 200)
    k, q = torch.zeros(2, 40, 64).bfloat16().cuda(), torch.zeros(1, 8, 64).bfloat16().cuda()
    layer.admit(0, k, k)
    out = torch.zeros(1, 8, 64, device="cuda")
    spans = [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in (layer.k_pages, layer.v_pages)]
    size = layer.k_pages.nbytes
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer.step(q, k[None, :, 0], k[None, :, 0], out=out)
        torch.cuda._sleep(20_000_000)
    del layer
    for _ in range(8):
        x = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert all(x.data_ptr() + size <= a or b <= x.data_ptr() for a, b in spans)
    torch.cuda.synchronize()
