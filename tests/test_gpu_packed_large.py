"""Packed causal attention on the GPU where keys, values or sequences are many:
heads one behind the other, rounds of head groups, lists in global memory, bins of
several lengths."""
import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402
from tests.test_gpu_packed import case, sa  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def test_more_keys_and_values_than_stay_in_l2(sa):  # noqa: F811
    # 8900 keys and values of 16 heads: 73 MB, so tiles go KV head by KV head
    lens = [4100, 1, 0, 2300, 129, 2040, 330]
    case(sa, 70, lens, lens, 16, 16, 128, pad=3)


@pytest.mark.parametrize("hq,hkv,d,lens_k", [
    (16, 16, 128, [9000, 5100, 4200]),      # 150 MB: several rounds, a head of them each
    (24, 12, 128, [9000, 9100, 6200]),      # 12 groups: a number of rounds that divides them
    (12, 12, 64, [15000, 14100, 3200])])
def test_rounds_of_head_groups(sa, hq, hkv, d, lens_k):  # noqa: F811
    # (keys count for rounds where a sequence has several tiles; one has a single one)
    case(sa, 71, [257, 300, 7], lens_k, hq, hkv, d, pad=2)


def test_a_call_of_rounds_behind_one_without(sa):  # noqa: F811
    # the same workspace: partial states of a round lie behind those of another
    att = sa.PackedAttention(16, 16, 128)
    for a, b in (([300, 200], [9000, 8000]), ([40, 30], [600, 500]), ([300, 200], [9000, 8000])):
        q, k, v, cq, ck = tp.inputs(72, a, b, 16, 16, 128, device="cuda")
        lse = torch.zeros(q.shape[:2], device="cuda")
        out = att(q, k, v, cq, ck, lse=lse)
        tp.check(tp.reference(q, k, v, cq, ck), out, lse, a, b, 128)
    assert int(att.dev_status.item()) == 0


def test_more_sequences_than_shared_memory_holds_with_more_keys_than_queries(sa):  # noqa: F811
    lens_q = [(5 * i) % 4 for i in range(1300)]
    lens_k = [n + (37 * i) % 300 for i, n in enumerate(lens_q)]
    case(sa, 73, lens_q, lens_k, 8, 2, 64, pad=4)


@pytest.mark.parametrize("lens_q,lens_k", [([1200, 131100], [1200, 131100]), ([3, 500], [600, 131500])])
def test_bins_of_several_lengths(sa, lens_q, lens_k):  # noqa: F811
    # from 131072 keys on a bin of the list holds tiles of several lengths; whole prompts, and chunks in shares
    q, k, v, cq, ck = tp.inputs(74, lens_q, lens_k, 1, 1, 64, device="cuda")
    att = sa.PackedAttention(1, 1, 64)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    att(q, k, v, cq, ck, out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(att.dev_status.item()) == 0
    # (the first sequence whole; of the second its first and last queries, and some between)
    n, m = lens_q[1], lens_k[1]
    rows = sorted({*range(min(n, 40)), *range(n - min(n, 300), n), *range(0, n, 997)})
    first = lens_q[0]
    tp.check(tp.reference(q[:first], k[:lens_k[0]], v[:lens_k[0]], tp.cu_of(lens_q[:1]), tp.cu_of(lens_k[:1])),
             out[:first], lse[:first], lens_q[:1], lens_k[:1], 64)
    for r in rows:
        seen = r + m - n + 1
        at = slice(first + r, first + r + 1)
        kk, vv = k[lens_k[0]:lens_k[0] + seen], v[lens_k[0]:lens_k[0] + seen]
        tp.check(tp.reference(q[at], kk, vv, tp.cu_of([1]), tp.cu_of([seen])), out[at], lse[at], [1], [seen], 64)
