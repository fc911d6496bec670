"""Pages, rotary positions, packed attention and the paged cache together, as a
server would run them: prompts admitted together, then captured decode steps,
sequences that end and others that take their places."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import packed as opk  # noqa: E402
from oracle import paged as op  # noqa: E402
from oracle import rotary as orot  # noqa: E402
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


def f64(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Server:
    """One layer: what a user of the operators writes."""

    def __init__(self, sa, batch, hq, hkv, d, page, pages, max_pages, weights):
        bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
        slots = (batch, hkv, max_pages * page)
        self.cache = sa.PagedCache(
            torch.zeros(pages, page, d, **bf), torch.zeros(pages, page, d, **bf),
            torch.zeros(batch, hkv, max_pages, **i32), torch.zeros(batch, hkv, **i32),
            weights=torch.zeros(slots, device="cuda") if weights else None,
            positions=torch.zeros(slots, **i32) if weights else None, num_q_heads=hq)
        self.pool = sa.PagePool.of(self.cache)
        self.rotary = sa.Rotary(d, rot_dim=d // 2, interleaved=True, base=500000.0)
        self.attention = sa.PackedAttention(hq, hkv, d, tokens=2000, batch=batch)
        self.start, self.hq, self.hkv, self.batch = torch.zeros(batch, **i32), hq, hkv, batch
        self.ended = torch.zeros(batch, dtype=torch.bool, device="cuda")
        self.counts = torch.zeros(batch, **i32)

    def prompts(self, q, k, v, cu):
        t = q.shape[0]
        slots = torch.empty(self.hkv, t, dtype=torch.int64, device="cuda")
        pos = torch.empty(t, dtype=torch.int32, device="cuda")
        self.pool.grow(slots, cu=cu, ended=self.ended, start=self.start, positions=pos)
        self.ended.zero_()
        q, k = self.rotary.store(q, k, v, pos, self.cache, slots, k_out=torch.empty_like(k))
        return self.attention(q, k, v, cu, out=torch.zeros_like(q))

    def step(self, q, k, v, out):
        slots = torch.empty(self.hkv, self.batch, dtype=torch.int64, device="cuda")
        pos = torch.empty(self.batch, dtype=torch.int32, device="cuda")
        self.pool.grow(slots, counts=self.counts, start=self.start, positions=pos)
        q, _ = self.rotary.store(q, k, v, pos, self.cache, slots)
        self.cache.attend(q, out=out)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 64, 16), (28, 4, 128, 32)])
def test_prompts_then_captured_steps(sa, hq, hkv, d, page, weights):
    batch = 3
    s = Server(sa, batch, hq, hkv, d, page, 200, 20, weights)
    g = torch.Generator().manual_seed(1)
    rot = s.rotary

    def tokens(n):
        x = torch.randn(n, hq + 2 * hkv, d, generator=g).bfloat16().cuda()
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    history = [[] for _ in range(batch)]          # per sequence: rotated keys and values as they were rounded

    def turned(x, positions):
        return torch.tensor(orot.rotate(f64(x), positions, rot.frequencies, rot.factor, rot.interleaved))

    def note(b, k, v, first):
        kk = rot(k, k, torch.arange(first, first + k.shape[0], dtype=torch.int32, device="cuda"))[1]
        # (rotated on its own: within the rounding of the formula)
        ref = turned(k, np.arange(first, first + k.shape[0]))
        assert (kk.double().cpu() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 1e-5
        history[b].append((f64(kk), f64(v)))

    lens = [0, 45, 130]
    q, k, v = tokens(sum(lens))
    cu = tp.cu_of(lens).cuda()
    out = s.prompts(q, k, v, cu)
    at = 0
    for b, n in enumerate(lens):
        if n:
            note(b, k[at:at + n], v[at:at + n], 0)
        at += n
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    rq, rk = rot(q, k, pos)
    tp.check(tp.reference(rq, rk, v, cu, cu), out, None, lens, lens, d)

    # decode steps of the two active sequences, captured
    s.counts.copy_(torch.tensor([0, 1, 1], dtype=torch.int32))
    sq, sk, sv = (t.clone() for t in tokens(batch))
    o = torch.zeros(batch, hq, d, device="cuda")
    state = [t.clone() for t in (s.cache.k_pages, s.cache.v_pages, s.cache.table, s.cache.lens, s.pool.owned,
                                 s.pool.free_pages, s.pool.free_count, s.start)]
    extra = [] if not weights else [t.clone() for t in (s.cache.weights, s.cache.positions)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step(sq, sk, sv, o)                     # a first run outside the graph, undone
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step(sq, sk, sv, o)
    for t, x in zip((s.cache.k_pages, s.cache.v_pages, s.cache.table, s.cache.lens, s.pool.owned, s.pool.free_pages,
                     s.pool.free_count, s.start), state):
        t.copy_(x)
    if weights:
        s.cache.weights.copy_(extra[0])
        s.cache.positions.copy_(extra[1])

    def check_step():
        pools = f64(s.cache.k_pages), f64(s.cache.v_pages)
        table, held = f64(s.cache.table), f64(s.cache.lens)
        first = [sum(x[0].shape[0] for x in history[b]) for b in range(batch)]
        for b in range(batch):
            if int(s.counts[b]):
                note(b, sk[b:b + 1], sv[b:b + 1], first[b])
        p = torch.tensor(first, dtype=torch.int32, device="cuda")
        rq = rot(sq, sk, p)[0]
        got = f64(o)
        for b in range(batch):
            if not history[b]:
                assert (got[b] == 0).all() and (held[b] == 0).all()
                continue
            kk, vv = (np.concatenate([x[i] for x in history[b]]) for i in (0, 1))
            n = kk.shape[0]
            assert (held[b] == n).all() and int(s.start[b]) == n
            for h in range(hkv):                  # every token is where the table says
                pg, x = op.slot_rows(table[b, h], np.arange(n), page)
                np.testing.assert_array_equal(pools[0][pg, x], kk[:, h])
                np.testing.assert_array_equal(pools[1][pg, x], vv[:, h])
            if int(s.counts[b]):
                ref, _, absv, absqk = opk.attend(f64(rq[b:b + 1]), kk, vv, [0, 1], [0, n])
                # attend's bound for fp32 output: scores off by E, three parts of a weight
                e = 2 * absqk[..., None] * (d + 8) * 2.0 ** -23 + 2.0 ** -16 + 2.0 ** -20 + n * 2.0 ** -23
                assert (np.abs(got[b] - ref[0]) <= e[0] * absv[0] + 2.0 ** -24 * np.abs(ref[0]) + 1e-30).all()

    for _ in range(20):
        for t, x in zip((sq, sk, sv), tokens(batch)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check_step()

    # sequence 1 ends and another prompt takes its place; the empty one gets its first
    s.ended.copy_(torch.tensor([False, True, False]))
    lens = [33, 70, 0]
    q, k, v = tokens(sum(lens))
    cu = tp.cu_of(lens).cuda()
    free = int(s.pool.free_count)
    out = s.prompts(q, k, v, cu)
    old = len(history[1]) and sum(x[0].shape[0] for x in history[1])
    history[1] = []
    note(0, k[:33], v[:33], 0)
    note(1, k[33:], v[33:], 0)
    pages = lambda n: -(-n // page)  # noqa: E731
    assert int(s.pool.free_count) == free + hkv * (pages(old) - pages(33) - pages(70))
    s.counts.fill_(1)
    for _ in range(5):
        for t, x in zip((sq, sk, sv), tokens(batch)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check_step()
    if weights:                                   # rows cut by an eviction give their pages back at the next step
        s.cache.evict([48] * hkv, sinks=4, recent=16)
        free = int(s.pool.free_count)
        held = f64(s.cache.lens)
        before = f64(s.pool.owned)
        graph.replay()
        torch.cuda.synchronize()
        need = -(-(held + 1) // page)
        np.testing.assert_array_equal(f64(s.pool.owned), need)
        assert int(s.pool.free_count) == free + int((before - need).sum())
        pos = f64(s.cache.positions)
        for b in range(batch):
            for h in range(hkv):
                n = int(held[b, h]) + 1
                assert len(set(pos[b, h, :n])) == n and pos[b, h, n - 1] == int(s.start[b]) - 1
    for x in (s.cache, s.pool, s.rotary, s.attention):
        assert int(x.dev_status.item()) == 0


FIRST_CALLS = """
import torch, head_heterogeneous_block_gb300 as sa
def captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    torch.cuda.synchronize()
    return graph, out
torch.zeros(1, device="cuda")
make = lambda *s: torch.randn(*s, device="cuda").bfloat16()
i32 = dict(dtype=torch.int32, device="cuda")
for d, nq, nk in ((64, 300, 300), (128, 3000, 9000)):
    q, k, cu = make(nq, 8, d), make(nk, 2, d), torch.tensor([0, 100, 300], **i32)
    attention = sa.PackedAttention(8, 2, d)
    graph, out = captured(lambda: attention(q, k, k, cu * (nq // 300), cu * (nk // 300)))
    again = attention(q, k, k, cu * (nq // 300), cu * (nk // 300))
    assert torch.equal(out, again) and int(attention.dev_status.item()) == 0
rotary, positions = sa.Rotary(128), torch.arange(3000, **i32)
graph, (a, b) = captured(lambda: rotary(q, k[:3000], positions))
assert torch.equal(a, rotary(q, k[:3000], positions)[0])
table, lens = torch.zeros(2, 2, 32, **i32), torch.zeros(2, 2, **i32)
pool = sa.PagePool(table, lens, 16, num_pages=100)
slots = torch.zeros(2, 300, dtype=torch.int64, device="cuda")
graph, _ = captured(lambda: pool.grow(slots, cu))
assert lens.tolist() == [[100, 100], [200, 200]] and int(pool.dev_status.item()) == 0
assert len(set(slots.flatten().tolist())) == 600 and int(pool.free_count.item()) == 100 - 2 * 7 - 2 * 13
print("right")
"""


def test_the_first_calls_of_a_process_may_be_captured(sa):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "right", r.stderr[-2000:]
