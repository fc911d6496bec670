"""Packed causal attention on the GPU against the oracle."""
import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import head_heterogeneous_block_gb300 as sa
    return sa


def run(sa, hq, hkv, d, q, k, v, cq, ck, with_lse=True, scale=None):
    att = sa.PackedAttention(hq, hkv, d, scale=scale)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=q.device) if with_lse else None
    got = att(q, k, v, cq, ck, out=out, lse=lse)
    assert got is out
    torch.cuda.synchronize()
    assert int(att.dev_status.item()) == 0
    return out, lse


def case(sa, seed, lens_q, lens_k, hq, hkv, d, pad=0, sharp=1.0, with_lse=True, scale=None):
    q, k, v, cq, ck = tp.inputs(seed, lens_q, lens_k, hq, hkv, d, pad, sharp, "cuda")
    out, lse = run(sa, hq, hkv, d, q, k, v, cq, ck, with_lse, scale)
    tp.check(tp.reference(q, k, v, cq, ck, scale), out, lse, lens_q, lens_k, d)
    if pad:
        assert (out[sum(lens_q):] == 7.0).all()
        assert lse is None or (lse[sum(lens_q):] == 7.0).all()


# one tile a CTA, no schedule: one token, part of a tile, several tiles, empty sequences among them
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (28, 4, 128), (4, 4, 64)])
@pytest.mark.parametrize("lens", [[1], [41], [64], [129], [0, 5, 0, 33, 1, 0]])
def test_small(sa, lens, hq, hkv, d):
    case(sa, 1, lens, lens, hq, hkv, d, pad=3)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (28, 4, 128), (16, 16, 64), (12, 1, 128), (22, 2, 128),
                                      (32, 2, 64), (6, 2, 128), (1, 1, 128)])
@pytest.mark.parametrize("lens", [[300, 1, 0, 700, 129, 64], [1030]])
def test_ragged(sa, lens, hq, hkv, d):
    case(sa, 2, lens, lens, hq, hkv, d, pad=5)


@pytest.mark.parametrize("lens_q,lens_k", [([17, 1, 130], [900, 257, 130]), ([1], [5000]), ([20, 3], [6000, 40]),
                                           ([5] * 9, [1, 2, 5, 6, 129, 1000, 0, 3, 4])])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (28, 4, 128)])
def test_more_or_fewer_keys_than_queries(sa, lens_q, lens_k, hq, hkv, d):
    case(sa, 3, lens_q, lens_k, hq, hkv, d)


def test_many_short_sequences(sa):
    lens = [(7 * i) % 40 for i in range(1500)]
    case(sa, 4, lens, lens, 8, 2, 64, pad=1)


def test_a_long_prompt(sa):
    case(sa, 5, [4099], [4099], 8, 2, 128)


def test_without_lse_and_with_a_scale(sa):
    case(sa, 6, [200, 77], [300, 77], 8, 2, 128, with_lse=False)
    case(sa, 6, [200, 77], [300, 77], 8, 2, 64, scale=0.31)


def test_no_keys_at_all(sa):
    case(sa, 7, [5, 40], [0, 0], 8, 2, 64)


def test_no_queries_at_all(sa):
    q, k, v, cq, ck = tp.inputs(8, [0, 0], [4, 6], 8, 2, 64, device="cuda")
    out, lse = run(sa, 8, 2, 64, q, k, v, cq, ck)
    assert out.numel() == 0 and lse.numel() == 0


# scores far above the first block's: sums near and beyond 2^126 (the careful pass), in whole and cut tiles
@pytest.mark.parametrize("lens_q,lens_k", [([600], [600]), ([20], [4000]), ([1, 700, 40], [300, 900, 2500])])
@pytest.mark.parametrize("sharp", [20.0, 200.0])
def test_wide_scores(sa, lens_q, lens_k, sharp):
    case(sa, 9, lens_q, lens_k, 8, 2, 128, sharp=sharp)


@pytest.mark.parametrize("power", [60, 115, 125, 140, 4000])
def test_a_late_key_above_the_first_block(sa, power):
    # key 400 scores `power` (base 2) for every query, the others about 0
    n, d = 600, 64
    q, k, v, cq, ck = tp.inputs(10, [n], [n], 2, 1, d, device="cuda")
    q[..., 0] = 8.0
    k[..., 0] = 0.0
    k[400] = 0.0
    k[400, :, 0] = power * 0.6931471805599453
    out, lse = run(sa, 2, 1, d, q, k, v, cq, ck)
    tp.check(tp.reference(q, k, v, cq, ck), out, lse, [n], [n], d)


def test_what_a_query_does_not_see_never_reaches_it(sa):
    lens_q, lens_k = [150, 40, 20], [150, 300, 20]
    q, k, v, cq, ck = tp.inputs(11, lens_q, lens_k, 8, 2, 128, pad=9, device="cuda")
    ref, lse_ref = run(sa, 8, 2, 128, q, k, v, cq, ck)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda").bfloat16()
    # behind the last sequence, and the later tokens of one and of another
    for t in (k, v):
        t[470:] = bad[torch.randint(0, 4, t[470:].shape, device="cuda")]
        t[100:150] = bad[torch.randint(0, 4, t[100:150].shape, device="cuda")]
        t[449] = bad[0]
    q[210:] = bad[0]
    out, lse = run(sa, 8, 2, 128, q, k, v, cq, ck)
    clean = torch.ones(219, dtype=torch.bool, device="cuda")
    clean[100:150] = False            # sees the first sequence's bad keys
    clean[182:190] = False            # one of them sees the second's last key, the others share its tile
    clean[210:] = False
    tp.same(out[clean.nonzero()[:, 0]], ref[clean.nonzero()[:, 0]])
    tp.same(lse[clean.nonzero()[:, 0]], lse_ref[clean.nonzero()[:, 0]])
    assert out[100:150].isnan().all() and out[189].isnan().all()
    # done again with their true maxima: the same up to the weights' rounding
    assert (out[182:189] - ref[182:189]).float().abs().max() <= 2.0 ** -6 * v[150:449].float().abs().max()
    assert (lse[182:189] - lse_ref[182:189]).abs().max() <= 2.0 ** -14


def test_infinities_and_nan_that_queries_see(sa):
    n, d = 300, 64
    q, k, v, cq, ck = tp.inputs(12, [n], [n], 4, 2, d, device="cuda")
    ref, _ = run(sa, 4, 2, d, q, k, v, cq, ck)
    v[170, 0, 3] = float("inf")
    v[200, 0, 3] = -float("inf")
    v[180, 1, 5] = float("nan")
    out, _ = run(sa, 4, 2, d, q, k, v, cq, ck)
    assert (out[170:200, :2, 3] == float("inf")).all() and out[200:, :2, 3].isnan().all()
    assert out[180:, 2:, 5].isnan().all()
    same = torch.ones_like(out, dtype=torch.bool)
    same[170:, :2, 3] = False
    same[180:, 2:, 5] = False
    # (the item is done again with its true maxima: not the same bits)
    assert torch.isfinite(out[same]).all()
    err = (out - ref).float().abs()[same]
    assert (err <= 2.0 ** -6 * v.float().abs().nan_to_num(0, 0, 0).max()).all()


@pytest.mark.parametrize("d", [64, 128])
def test_layouts(sa, d):
    lens = [130, 70]
    q, k, v, cq, ck = tp.inputs(13, lens, lens, 8, 2, d, device="cuda")
    ref, _ = run(sa, 8, 2, d, q, k, v, cq, ck)
    att = sa.PackedAttention(8, 2, d)
    fused = torch.cat((q, k, v), 1)
    tp.same(att(fused[:, :8], fused[:, 8:10], fused[:, 10:], cq), ref)
    head_major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    out = torch.empty(8, 200, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    tp.same(att(*head_major, cq, out=out).contiguous(), ref)
    wide = torch.zeros(200, 8, d + 8, dtype=torch.bfloat16, device="cuda")
    wide[..., :d] = q
    tp.same(att(wide[..., :d], k, v, cq), ref)


def test_same_bits_again(sa):
    lens_q, lens_k = [40, 900, 3], [4000, 900, 2000]
    q, k, v, cq, ck = tp.inputs(14, lens_q, lens_k, 8, 2, 128, sharp=30.0, device="cuda")
    first = run(sa, 8, 2, 128, q, k, v, cq, ck)
    for _ in range(5):
        again = run(sa, 8, 2, 128, q, k, v, cq, ck)
        tp.same(again[0], first[0])
        tp.same(again[1], first[1])


def test_a_captured_call_follows_the_lengths(sa):
    hq, hkv, d, total = 8, 2, 64, 900
    att = sa.PackedAttention(hq, hkv, d, tokens=total, batch=3)
    q, k, v, cq, ck = tp.inputs(15, [300, 0, 600], [300, 0, 600], hq, hkv, d, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(total, hq, device="cuda")
    att(q, k, v, cq, ck, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att(q, k, v, cq, ck, out=out, lse=lse)
    for lens in ([300, 0, 600], [1, 2, 3], [900, 0, 0], [0, 0, 0], [449, 450, 1]):
        cq.copy_(tp.cu_of(lens))
        ck.copy_(tp.cu_of(lens))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        tp.check(tp.reference(q, k, v, cq, ck), out, lse, lens, lens, d)
        assert (out[sum(lens):] == 7.0).all()
    assert int(att.dev_status.item()) == 0


def test_on_another_stream(sa):
    lens = [200, 500]
    q, k, v, cq, ck = tp.inputs(16, lens, lens, 8, 2, 64, device="cuda")
    ref, _ = run(sa, 8, 2, 64, q, k, v, cq, ck)
    att = sa.PackedAttention(8, 2, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = att(q, k, v, cq, ck, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    tp.same(out, ref)
    out = att(q, k, v, cq, ck, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    tp.same(out, ref)


@pytest.mark.parametrize("ends", [[0, 50, 20, 100], [0, 50, 60, 4000], [-7, 50, 60, 100], [9, 9, 2, -1],
                                  [2 ** 31 - 1, -2 ** 31, 5, 100]])
@pytest.mark.parametrize("total", [100, 1600])
def test_bad_lengths_are_clamped_and_flagged(sa, ends, total):
    q, k, v, cq, _ = tp.inputs(17, [total], [total], 8, 2, 64, device="cuda")
    att = sa.PackedAttention(8, 2, 64)
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 50, 60, 100], dtype=torch.int32, device="cuda")
    for a, b in ((cu, good), (good, cu), (cu, cu)):
        att.dev_status.zero_()
        out = torch.full_like(q, 7.0)
        att(q, k, v, a, b, out=out)
        torch.cuda.synchronize()
        assert int(att.dev_status.item()) == sa.SA_DEV_BAD_COUNT
    att.dev_status.zero_()
    tp.same(att(q, k, v, cq), run(sa, 8, 2, 64, q, k, v, cq, cq)[0])
    assert int(att.dev_status.item()) == 0


def test_a_wait_that_runs_out(sa):
    lens = [700]
    q, k, v, cq, ck = tp.inputs(18, lens, lens, 8, 2, 128, device="cuda")
    ref, _ = run(sa, 8, 2, 128, q, k, v, cq, ck)
    att = sa.PackedAttention(8, 2, 128)
    sa.sparse_attn_set_wait_limit(100)
    try:
        att(q, k, v, cq, ck)
        torch.cuda.synchronize()
        assert int(att.dev_status.item()) == sa.SA_DEV_TIMEOUT
    finally:
        sa.sparse_attn_set_wait_limit(0)
    att.dev_status.zero_()
    tp.same(att(q, k, v, cq, ck), ref)
    assert int(att.dev_status.item()) == 0


def test_more_items_than_a_batch_of_a_cta(sa):
    # one token a sequence: the output is its value; some values are infinite, so that their items are done again
    n, heads, d = 6000, 16, 64
    q, k, v, cq, ck = tp.inputs(20, [1] * n, [1] * n, heads, heads, d, device="cuda")
    v[::37, 3, 5] = float("inf")
    v[::41, 7, 9] = float("nan")
    out, lse = run(sa, heads, heads, d, q, k, v, cq, ck)
    assert torch.equal(out.nan_to_num(7.0, 8.0, 9.0), v.nan_to_num(7.0, 8.0, 9.0))
    ref = (q.double() * k.double()).sum(-1) / d ** 0.5
    bound = (q.double() * k.double()).abs().sum(-1) / d ** 0.5 * (d + 8) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * ref.abs()
    assert ((lse.double() - ref).abs() <= bound).all()


def test_calls_of_other_sizes_one_behind_the_other(sa):
    # one workspace, several of its sizes, schedules and joins, without a synchronisation between
    att = sa.PackedAttention(8, 2, 64)
    todo = [([41], [41]), ([700, 3, 300], [700, 3, 300]), ([20, 5], [6000, 900]), ([1] * 40, [33] * 40), ([2000], [2000]),
            ([64], [4000]), ([0, 7], [0, 7])]
    cases = [tp.inputs(30 + i, a, b, 8, 2, 64, device="cuda") for i, (a, b) in enumerate(todo)]
    lse = [torch.zeros(x[0].shape[:2], device="cuda") for x in cases]
    for _ in range(3):
        outs = [att(*x, lse=y) for x, y in zip(cases, lse)]
    torch.cuda.synchronize()
    assert int(att.dev_status.item()) == 0
    for x, o, y, (a, b) in zip(cases, outs, lse, todo):
        tp.check(tp.reference(*x), o, y, a, b, 64)


def test_a_workspace_that_grows(sa):
    att = sa.PackedAttention(8, 2, 64)
    made = set()
    for n in (1, 50, 300, 301, 302, 5000, 9000, 9001):
        q, k, v, cq, ck = tp.inputs(40 + n % 7, [n], [n], 8, 2, 64, device="cuda")
        tp.same(att(q, k, v, cq), run(sa, 8, 2, 64, q, k, v, cq, ck)[0])
        made.add(att._ws_ptr)
    assert len(made) <= 3 and int(att.dev_status.item()) == 0


@pytest.mark.parametrize("lens_q,lens_k", [([60], [60]), ([600, 40], [600, 40]), ([20], [4000]), ([1, 700, 40], [300, 900, 2500])])
@pytest.mark.parametrize("masked", [False, True])
def test_values_near_the_end_of_the_range(sa, lens_q, lens_k, masked):
    # the mean of such values is finite, their sum is not; a NaN that the first sequence's last queries alone see
    q, k, v, cq, ck = tp.inputs(50, lens_q, lens_k, 8, 2, 128, device="cuda")
    v = (v.float() * 1.2e38).clamp(-3.3e38, 3.3e38).bfloat16()
    ref = tp.reference(q, k, v, cq, ck)
    seen = 0
    if masked:
        v[lens_k[0] - 1] = float("nan")
        seen = lens_q[0]                  # (NaN in the last one of these only)
    out, lse = run(sa, 8, 2, 128, q, k, v, cq, ck)
    if masked:
        assert out[seen - 1].isnan().all()
        out[seen - 1], lse[seen - 1] = (torch.from_numpy(x[seen - 1]).cuda().to(t.dtype) for x, t in zip(ref, (out, lse)))
    tp.check(ref, out, lse, lens_q, lens_k, 128)


@pytest.mark.parametrize("power", [60, 115])
def test_large_values_behind_a_late_key(sa, power):
    # the late key's weight times its values overflows, and the sum of weights does not
    n, d = 600, 64
    q, k, v, cq, ck = tp.inputs(10, [n], [n], 2, 1, d, device="cuda")
    q[..., 0] = 8.0
    k[..., 0] = 0.0
    k[400] = 0.0
    k[400, :, 0] = power * 0.6931471805599453
    v = (v.float() * 2.0 ** 90).bfloat16()
    out, lse = run(sa, 2, 1, d, q, k, v, cq, ck)
    tp.check(tp.reference(q, k, v, cq, ck), out, lse, [n], [n], d)


def test_two_objects_on_two_streams_at_once(sa):
    # each with its workspace: lists, shares and joins of both under way together
    todo = [([700, 3, 300], [700, 3, 300]), ([20, 5], [6000, 900])]
    cases = [tp.inputs(60 + i, a, b, 8, 2, 128, device="cuda") for i, (a, b) in enumerate(todo)]
    refs = [run(sa, 8, 2, 128, *x) for x in cases]
    atts = [sa.PackedAttention(8, 2, 128) for _ in todo]
    streams = [torch.cuda.Stream() for _ in todo]
    torch.cuda.synchronize()
    outs = [[] for _ in todo]
    for _ in range(20):
        for i, (x, att, s) in enumerate(zip(cases, atts, streams)):
            with torch.cuda.stream(s):
                outs[i].append(att(*x))
    torch.cuda.synchronize()
    for i, (ref, att) in enumerate(zip(refs, atts)):
        assert int(att.dev_status.item()) == 0
        for o in outs[i]:
            tp.same(o, ref[0])


def test_items_of_every_length_in_turn(sa):
    # short items between long ones: Q comes from shared memory, from tensor memory and from both in turn
    lens = [130, 1500, 40, 600, 129, 2000, 500, 5, 385, 900, 512, 513]
    case(sa, 61, lens, lens, 4, 4, 128)
    case(sa, 62, lens, [n + 300 * (i % 3) for i, n in enumerate(lens)], 32, 4, 128)
    case(sa, 63, lens, lens, 4, 4, 64)
