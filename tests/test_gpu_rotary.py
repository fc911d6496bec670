"""Rotary positions on the GPU against the oracle.

Tolerance.  An angle is off by at most 2^-24 half turns (pi 2^-24 radians) and
position * 2^-65 turns; sine and cosine add 2^-22, their product with the factor
2^-23, the two products and their sum 2^-22 of the pair's |x| + |y|: together
below 2^-20 (|x| + |y|) |factor|.  The value then rounds to bf16: 2^-8 of it.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import rotary as orot  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa


def f64(t):
    return t.double().cpu().numpy()


def check(rot, x, positions, got):
    x = f64(x)
    ref = orot.rotate(x, positions.cpu().numpy(), rot.frequencies, rot.factor, rot.interleaved)
    n, r = x.shape, rot.rot_dim
    size = np.zeros(n)
    a = np.abs(x[..., :r])
    pair = a.reshape(*n[:2], r // 2, 2).sum(-1).repeat(2, -1) if rot.interleaved else \
        np.concatenate([a[..., :r // 2] + a[..., r // 2:]] * 2, -1)
    size[..., :r] = pair * abs(rot.factor)
    g = f64(got)
    assert (np.abs(g - ref) <= 2.0 ** -20 * size + 2.0 ** -8 * np.abs(ref)).all()
    assert (g[..., r:] == x[..., r:]).all()


def inputs(seed, tokens, hq, hkv, d, fused=False, far=1000):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(tokens, hq + 2 * hkv, d, generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q, k, v, torch.randint(0, far, (tokens,), generator=g).int().cuda()


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112), (128, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 8, 2), (3, 28, 4), (70, 5, 5), (2500, 7, 1)])
def test_rotary(sa, tokens, hq, hkv, d, rot, interleaved):
    r = sa.Rotary(d, rot_dim=rot, interleaved=interleaved)
    for fused in (False, True):
        q, k, v, pos = inputs(1, tokens, hq, hkv, d, fused)
        before = q.clone(), k.clone()
        qo, ko = r(q, k, pos)
        torch.cuda.synchronize()
        check(r, q, pos, qo)
        check(r, k, pos, ko)
        assert torch.equal(q, before[0]) and torch.equal(k, before[1])
        r(q, k, pos, q_out=q, k_out=k)
        assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("scaling", [
    {"type": "linear", "factor": 4}, {"type": "ntk", "factor": 8},
    {"type": "wavelength", "factor": 8, "low": 1, "high": 4, "original": 8192},
    {"type": "yarn", "factor": 16, "original": 4096},
    {"type": "yarn", "factor": 4, "original": 32768, "beta_fast": 16, "beta_slow": 2, "attention_factor": 0.7}])
def test_scalings(sa, scaling):
    r = sa.Rotary(128, base=500000.0, scaling=scaling)
    q, k, v, pos = inputs(2, 300, 4, 2, 128, far=131072)
    qo, ko = r(q, k, pos)
    check(r, q, pos, qo)
    check(r, k, pos, ko)


def test_far_and_negative_positions(sa):
    r = sa.Rotary(64)
    q, k, v, _ = inputs(3, 9, 4, 2, 64)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 10 ** 6 + 7, 123456789, -98765], dtype=torch.int32,
                       device="cuda")
    qo, ko = r(q, k, pos)
    # fp64 angles of positions of 2^31 are themselves off by 2^-22: these by exact integers
    turns = [int(t) % 2 ** 64 for t in r.turns.tolist()]
    exact = np.array([[(((int(p) * t) + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 * 2 * np.pi for t in turns]
                      for p in pos.tolist()])
    x = f64(q)
    a = exact[:, None, :]
    ref = np.concatenate([x[..., :32] * np.cos(a) - x[..., 32:] * np.sin(a),
                          x[..., 32:] * np.cos(a) + x[..., :32] * np.sin(a)], -1)
    size = np.concatenate([np.abs(x[..., :32]) + np.abs(x[..., 32:])] * 2, -1)
    assert (np.abs(f64(qo) - ref) <= 2.0 ** -20 * size + 2.0 ** -8 * np.abs(ref)).all()
    assert torch.equal(qo[0], q[0])


def test_infinities_and_nan_stay_in_their_pair(sa):
    r = sa.Rotary(64)
    q, k, v, pos = inputs(4, 40, 4, 2, 64)
    ref, _ = r(q, k, pos)
    q[3, 1, 5], q[7, 2, 40] = float("nan"), float("inf")
    got, _ = r(q, k, pos)
    touched = torch.zeros_like(q, dtype=torch.bool)
    touched[3, 1, 5] = touched[3, 1, 37] = touched[7, 2, 8] = touched[7, 2, 40] = True
    assert torch.equal(got[~touched], ref[~touched])
    assert not torch.isfinite(got[touched].float()).any()


def test_layouts(sa):
    r = sa.Rotary(128, rot_dim=64, interleaved=True)
    q, k, v, pos = inputs(5, 130, 8, 2, 128)
    ref = r(q, k, pos)
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k)]
    qo = torch.zeros(8, 130, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ko = torch.zeros(130, 2, 136, dtype=torch.bfloat16, device="cuda")
    r(*hm, pos, q_out=qo, k_out=ko[..., :128])
    assert torch.equal(qo, ref[0]) and torch.equal(ko[..., :128], ref[1]) and (ko[..., 128:] == 0).all()
    one = k[:, :1].expand(130, 2, 128)               # one key head for two
    _, ko = r(q, one, pos)
    assert torch.equal(ko[:, 0], ref[1][:, 0]) and torch.equal(ko[:, 1], ref[1][:, 0])


def pools(seed, pages, page, d, interleaved):
    g = torch.Generator().manual_seed(seed)
    both = torch.randn((pages, 2, page, d) if interleaved else (2, pages, page, d), generator=g).bfloat16().cuda()
    return (both[:, 0], both[:, 1]) if interleaved else (both[0], both[1])


@pytest.mark.parametrize("tokens,hq,hkv,d,page", [(1, 8, 2, 64, 16), (64, 32, 8, 128, 16), (77, 28, 4, 128, 64),
                                                  (1500, 16, 16, 64, 256), (3000, 7, 1, 128, 32)])
@pytest.mark.parametrize("together", [False, True])
def test_store(sa, tokens, hq, hkv, d, page, together):
    r = sa.Rotary(d)
    q, k, v, pos = inputs(6, tokens, hq, hkv, d, fused=True)
    pages = hkv * (-(-tokens // page)) + 3
    kp, vp = pools(7, pages, page, d, together)
    table = torch.zeros(1, hkv, 4, dtype=torch.int32, device="cuda")
    cache = sa.PagedCache(kp, vp, table, torch.zeros(1, hkv, dtype=torch.int32, device="cuda"))
    g = torch.Generator().manual_seed(8)
    slots = torch.randperm(pages * page, generator=g)[:hkv * tokens].view(hkv, tokens).cuda()
    slots[:, torch.rand(tokens, generator=g) < 0.1] = -1
    want_k, want_v = kp.clone(), vp.clone()
    ref = r(q, k, pos)
    for x in range(hkv):
        has = slots[x] >= 0
        at = slots[x][has]
        want_k[at // page, at % page] = ref[1][has, x]
        want_v[at // page, at % page] = v[has, x]
    ko = torch.zeros_like(ref[1])
    qo, got = r.store(q, k, v, pos, cache, slots, k_out=ko)
    assert got is ko and torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    kp.copy_(torch.randn_like(kp))
    kp0 = kp.clone()
    _, none = r.store(q, k, v, pos, cache, slots)       # the cache's copy alone
    assert none is None
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    at = slots[slots >= 0]
    used[at // page, at % page] = True
    assert torch.equal(kp[used], want_k[used]) and torch.equal(kp[~used], kp0[~used])
    assert int(r.dev_status.item()) == 0


def test_bad_slots_are_flagged_and_store_nothing(sa):
    r = sa.Rotary(64)
    q, k, v, pos = inputs(9, 6, 4, 2, 64)
    kp, vp = pools(10, 5, 16, 64, False)
    cache = sa.PagedCache(kp, vp, torch.zeros(1, 2, 2, dtype=torch.int32, device="cuda"),
                          torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    slots = torch.full((2, 6), -1, dtype=torch.int64, device="cuda")
    slots[0, :4] = torch.tensor([80, 2 ** 40, -2, -2 ** 63], device="cuda")
    before = kp.clone(), vp.clone()
    qo, _ = r.store(q, k, v, pos, cache, slots)
    assert int(r.dev_status.item()) == sa.SA_DEV_BAD_INDEX
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])
    assert torch.equal(qo, r(q, k, pos)[0])


def test_no_tokens(sa):
    r = sa.Rotary(64)
    q, k, v, pos = inputs(11, 0, 4, 2, 64)
    qo, ko = r(q, k, pos)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)


def test_streams_and_graphs(sa):
    r = sa.Rotary(128)
    q, k, v, pos = inputs(12, 50, 8, 2, 128)
    ref = r(q, k, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = r(q, k, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r(q, k, pos, q_out=qo, k_out=ko)
    pos.add_(5)
    graph.replay()
    again = r(q, k, pos)
    assert torch.equal(qo, again[0]) and torch.equal(ko, again[1])
