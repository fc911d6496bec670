"""The paged cache operators on the GPU where calls meet their limits: waits
that give up, aliased arguments, bad pages, other streams and devices."""
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


def _q(torch, seed, b, hq, d):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(b, hq, d, generator=g).bfloat16()


def test_attend_of_short_sequences_ends_when_waits_give_up(env):
    # every tile is a segment's first and last, and the waits give up at
    # different tiles; each launch ends, and the next one is right
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(60, [1 + 37 * x % 120 for x in range(400)], 4, 128, 16)
    dev, cache = P.to_gpu(c, sa, with_weights=False)
    q = _q(torch, 50, 400, 32, 128)
    gq = q.cuda()
    out, lse = torch.empty(400, 32, 128, device="cuda"), torch.empty(400, 32, device="cuda")
    try:
        for limit in (1, 200, 500, 1000, 1500, 2000, 3000, 5000):
            sa.sparse_attn_set_wait_limit(limit)
            for _ in range(4):
                cache.attend(gq, out=out, lse=lse)
            torch.cuda.synchronize()
            if limit == 1:
                assert int(cache.dev_status.item()) & sa.SA_DEV_TIMEOUT
    finally:
        sa.sparse_attn_set_wait_limit(0)
    cache.dev_status.zero_()
    cache.attend(gq, out=out, lse=lse)
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, out, lse)


@pytest.mark.parametrize("Bt,hkv,T", [(1, 8, 1), (1, 8, 300), (70, 1, 1), (5, 1, 300), (1, 1, 1)])
@pytest.mark.parametrize("inplace", [True, False])
def test_append_at_the_old_lengths(env, Bt, hkv, T, inplace):
    # start is a view of the lengths (of one sequence, or with one KV head):
    # they are read before the new ones replace them, in place or in lens_out
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    lens = np.arange(40, 40 + Bt)
    c = P.random_cache(T, lens + T, hkv, 64, 32, junk=False)
    c["lens"] = torch.as_tensor(lens, dtype=torch.int32)[:, None].expand(-1, hkv).contiguous()
    dev, cache = P.to_gpu(c, sa)
    kn = torch.randn(Bt, hkv, T, 64, generator=torch.Generator().manual_seed(T)).bfloat16()
    out = dev["lens"] if inplace else dev["lens"] + 1000
    start = out[:, 0]
    assert start.is_contiguous() and start.data_ptr() == out.data_ptr()
    ref = op.append(P.f64(c["k"]), P.f64(c["v"]), c["table"].numpy(), c["lens"].numpy(), P.f64(kn),
                    P.f64(kn), [T] * Bt, start.cpu().numpy(), P.f64(c["weights"]),
                    c["positions"].numpy())
    cache.append(kn.cuda(), kn.cuda(), start=start, lens_out=None if inplace else out)
    assert int(cache.dev_status.item()) == 0
    assert np.array_equal(P.f64(dev["k"]), ref[0]) and np.array_equal(P.f64(dev["v"]), ref[1])
    assert np.array_equal(out.cpu().numpy(), ref[2])
    assert np.array_equal(dev["positions"].cpu().numpy(), ref[4])


@pytest.mark.parametrize("T", [1, 300])
def test_append_into_the_counts(env, T):
    # with one KV head the new lengths may replace the counts they come from
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(T, [50 + T, 3 + T, 90 + T], 1, 64, 32, junk=False)
    c["lens"] = torch.tensor([[50], [3], [90]], dtype=torch.int32)
    dev, cache = P.to_gpu(c, sa)
    counts = torch.tensor([T, 0, max(1, T - 1)], dtype=torch.int32, device="cuda")
    want = (dev["lens"][:, 0] + counts).tolist()
    kn = torch.randn(3, 1, T, 64, device="cuda").bfloat16()
    cache.append(kn, kn, counts=counts, lens_out=counts[:, None])
    assert int(cache.dev_status.item()) == 0
    assert counts.tolist() == want and dev["lens"].flatten().tolist() == [50, 3, 90]
    at, x = dev["table"][2, 0, (90 + counts[2] - 91) // 32].long(), (counts[2].item() - 1) % 32
    assert torch.equal(dev["k"][at, x], kn[2, 0, counts[2].item() - 91])
    two = P.to_gpu(P.random_cache(1, [50, 60], 2, 64, 32, junk=False), sa)[1]
    kn = torch.zeros(2, 2, 1, 64, device="cuda").bfloat16()
    with pytest.raises(sa.SparseAttnError):            # row (0, 1) would replace sequence 1's count
        two.append(kn, kn, counts=two.lens.view(-1)[1:3])


@pytest.mark.parametrize("cap_pages", [7, 300])            # moved by the row's CTA, and by a second launch
@pytest.mark.parametrize("inplace", [True, False])
def test_evict_leaves_slots_of_bad_pages_whole(env, cap_pages, inplace):
    # a token that cannot move, for its own page or the hole's, leaves the
    # hole's key, value, weight and position together
    from tests import _paged as P
    sa, torch = env
    n, keep = 200, 60
    c = P.random_cache(61, [n, n, n], 1, 64, 32, max_pages=cap_pages, junk=False)
    c["weights"][:] = torch.arange(c["weights"].shape[-1]).float()     # the last ones stay
    c["table"][0, 0, 1] = -3                       # holes 32 to 59
    c["table"][1, 0, 5] = c["k"].shape[0]          # sources 160 to 191
    dev, cache = P.to_gpu(c, sa)
    k0 = dev["k"].cpu()
    outs = {} if inplace else {"weights_out": torch.zeros_like(dev["weights"]),
                               "positions_out": torch.zeros_like(dev["positions"])}
    cache.evict([keep], 0, 0, **outs)
    torch.cuda.synchronize()
    assert int(cache.dev_status.item()) == sa.SA_DEV_BAD_INDEX
    w, pos = (outs["weights_out"], outs["positions_out"]) if not inplace else (dev["weights"], dev["positions"])
    k1 = dev["k"].cpu()
    assert dev["lens"].flatten().tolist() == [keep] * 3
    for b in range(3):
        for t in range(keep):                      # slot t takes the token of slot 140 + t
            s = 140 + t
            stays = (b == 0 and t >= 32) or (b == 1 and 160 <= s < 192)
            holds = t if stays else s
            assert w[b, 0, t].item() == holds and pos[b, 0, t].item() == holds
            page = c["table"][b, 0, t // 32].item()
            if 0 <= page < k0.shape[0]:
                was = c["table"][b, 0, holds // 32].item()
                assert torch.equal(k1[page, t % 32], k0[was, holds % 32])


def test_rows_too_long_for_eviction_still_attend(env):
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(62, [300, 77], 2, 64, 32, max_pages=262144 // 32 + 1)
    dev, cache = P.to_gpu(c, sa, num_q_heads=4)
    q = _q(torch, 51, 2, 4, 64)
    o = cache.attend(q.cuda())
    assert int(cache.dev_status.item()) == 0
    P.check_attend(c, q, o, None, dev["weights"])
    with pytest.raises(sa.SparseAttnError) as e:
        cache.evict([100, 100])
    assert e.value.status == 3 and torch.equal(dev["lens"].cpu(), c["lens"])


def test_paged_decode_layer_copies_its_budgets(env):
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    sa, torch = env
    keep = np.array([40.5, 60.0])
    layer = PagedDecodeLayer(1, 8, 2, 64, 16, 20, 200, keep=keep)
    keep[:] = 0
    k = torch.zeros(2, 100, 64, dtype=torch.bfloat16, device="cuda")
    layer.admit(0, k, k)
    assert layer.lens.tolist() == layer.book.lens == [[40, 60]]
    assert len(layer.book.free) == 20 - 3 - 4


def _reused(torch, address):
    """Whether the current stream's small allocations are given the address."""
    got = [torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(8192)]
    return any(x.data_ptr() == address for x in got)


def test_status_word_outlives_work_of_the_workspaces_stream(env):
    # the status word comes from one stream, the workspace from the first
    # attend on another; the cache is dropped with that stream at work
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(63, [700, 90], 2, 128, 32)
    q = _q(torch, 52, 2, 40, 128).cuda()
    for first in (None, 8):                        # the workspace made, or outgrown, there
        dev, cache = P.to_gpu(c, sa, with_weights=False, num_q_heads=first)
        before = cache._ws_bytes
        out = torch.empty(2, 40, 128, dtype=torch.bfloat16, device="cuda")
        address = cache.dev_status.data_ptr()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        cache.attend(q, out=out, stream=side)
        with torch.cuda.stream(side):
            torch.cuda._sleep(600_000_000)
        cache.attend(q, out=out, stream=side)
        assert cache._ws_bytes > before
        del cache
        assert not _reused(torch, address) and not side.query()
        torch.cuda.synchronize()


def test_layers_status_word_outlives_work_of_another_stream(env):
    # an admission on another stream ORs its status word into the layer's
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    sa, torch = env
    layer = PagedDecodeLayer(1, 8, 2, 64, 16, 20, 200)
    k = torch.zeros(2, 40, 64, dtype=torch.bfloat16, device="cuda")
    address = layer.cache.dev_status.data_ptr()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer.admit(0, k, k)
        torch.cuda._sleep(600_000_000)
    del layer
    assert not _reused(torch, address) and not side.query()
    torch.cuda.synchronize()


def test_streams_of_another_device_are_refused(env):
    from types import SimpleNamespace
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(64, [40], 2, 64, 16, max_pages=4)
    dev, cache = P.to_gpu(c, sa)
    state = {n: dev[n].clone() for n in ("lens", "weights", "positions")}
    other = SimpleNamespace(device_index=dev["k"].get_device() + 1, cuda_stream=0)
    q = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: cache.append(k, k, stream=other), lambda: cache.attend(q, stream=other),
                 lambda: cache.evict([10, 10], stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    torch.cuda.synchronize()
    for n, t in state.items():
        assert torch.equal(dev[n], t)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 5, 8, 9, 16, 17, 32, 40])
def test_fp32_outputs_have_all_parts_of_the_weights(env, G, d):
    # scores without an error to hide behind: see the bound's derivation
    from tests import _paged_fp32 as F
    sa, torch = env
    from tests import _paged as P
    for lens, hkv, unit in (([0, 1, 24, 64, 100, 128, 300, 1000], 2, 64), ([64, 24, 128, 1] * 40, 1, 128)):
        c, q = F.inputs(d + G, lens, hkv, G, d, 32)
        dev, cache = P.to_gpu(c, sa, with_weights=False)
        out = torch.empty(q.shape, device="cuda")
        cache.attend(q.cuda(), out=out)
        assert int(cache.dev_status.item()) == 0
        over = F.check(c, q, out, unit)
        assert (over <= 1).all(), over.max()
        assert (out[np.array(lens) == 0] == 0).all()


def test_binding_functions_give_what_the_class_gives(env):
    # the torch-free functions, on addresses and explicit strides
    from tests import _paged as P
    sa, torch = env
    c = P.random_cache(65, [[50, 200], [0, 77]], 2, 64, 16, max_pages=16, spare=50, junk=False)
    free = [x for x in range(c["k"].shape[0]) if x not in c["table"].flatten().tolist()]
    c["table"][c["table"] < 0] = torch.tensor(free[:int((c["table"] < 0).sum())], dtype=torch.int32)
    q = _q(torch, 53, 2, 8, 64).cuda()
    qkv = torch.randn(2, 3, 6, 64, device="cuda").bfloat16()
    k, v = qkv[:, :, 2:4].transpose(1, 2), qkv[:, :, 4:].transpose(1, 2)
    counts = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    start = torch.tensor([900, 800], dtype=torch.int32, device="cuda")
    states, outs = [], []
    for binding in (False, True):
        dev, cache = P.to_gpu(c, sa, num_q_heads=8)
        out, lse = torch.empty(2, 8, 64, device="cuda"), torch.empty(2, 8, device="cuda")
        if binding:
            d = cache.desc
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            need = max(sa.sparse_attn_paged_attend_workspace_size(d, 8, True),
                       sa.sparse_attn_paged_evict_workspace_size(d))
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            stream = torch.cuda.current_stream()
            sa.sparse_attn_paged_append(d, k.data_ptr(), v.data_ptr(), k.stride()[:3], v.stride()[:3],
                                        3, counts, start, dev["lens"], st, stream=stream)
            sa.sparse_attn_paged_attend(d, q.data_ptr(), *q.stride()[:2], 8, out, lse, dev["weights"],
                                        ws, need, st, stream=stream)
            sa.sparse_attn_paged_evict(d, [40, 60], 4, 8, dev["lens"], dev["weights"],
                                       dev["positions"], ws, need, st, stream=stream)
            assert int(st.item()) == 0
        else:
            cache.append(k, v, counts=counts, start=start)
            cache.attend(q, out=out, lse=lse)
            cache.evict([40, 60], 4, 8)
        assert int(cache.dev_status.item()) == 0
        torch.cuda.synchronize()
        states.append(dev)
        outs.append((out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert states[0]["lens"].tolist() == [[40, 60], [2, 60]]
    for n in states[0]:
        assert torch.equal(states[0][n], states[1][n]), n


def test_weights_that_an_admission_leaves(env):
    # each query attends over the whole prompt, later tokens included
    from head_heterogeneous_block_gb300.layer import PagedDecodeLayer
    from oracle import paged as op
    from tests import _paged as P
    sa, torch = env
    S, W, hkv, hq, d = 150, 5, 2, 8, 64
    g = torch.Generator().manual_seed(66)
    k, v = (torch.randn(hkv, S, d, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(W, hq, d, generator=g).bfloat16()
    layer = PagedDecodeLayer(2, hq, hkv, d, 16, num_pages=40, max_tokens=200, keep=[200, 200])
    layer.admit(1, k.cuda(), v.cuda(), queries=q.cuda())
    assert int(layer.cache.dev_status.item()) == 0 and layer.lens.tolist() == [[0, 0], [S, S]]
    got = P.f64(layer.weights)
    table, lens = np.arange(hkv, dtype=np.int32)[None, :, None], np.full((1, hkv), S, np.int32)
    want, tol = np.zeros((hkv, S)), np.zeros((hkv, S))
    for i in range(W):
        _, _, w, _, absqk = op.attend(P.f64(q[i:i + 1]), P.f64(k), P.f64(v), table, lens,
                                      np.zeros((1, hkv, S)))
        E = absqk[0].reshape(hkv, -1).max(1)[:, None] * (d + 8) * 2.0 ** -23
        want += w[0]
        tol += (2 * E + 2.0 ** -20 + S * 2.0 ** -23) * w[0]
    tol += W * 2.0 ** -22 * want                   # as many additions to the weight
    assert (np.abs(got[1, :, :S] - want) <= tol).all()
    assert (got[0] == 0).all() and (got[1, :, S:] == 0).all()
