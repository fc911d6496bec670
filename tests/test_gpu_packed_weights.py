"""Packed causal attention where the rounding of the weights has to cancel: rows of
one dominant key, wherever it is, and rows whose weights are all the same."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402
from tests.test_gpu_packed import sa  # noqa: E402, F401
from tests.test_gpu_packed_scores import LENS, check  # noqa: E402

pytestmark = pytest.mark.gpu


def run(sa, q, k, v, cq, ck, with_lse):  # noqa: F811
    att = sa.PackedAttention(q.shape[1], k.shape[1], q.shape[2])
    lse = torch.full(q.shape[:2], 7.0, device="cuda") if with_lse else None
    out = att(q, k, v, cq, ck, out=torch.full_like(q, 7.0), lse=lse)
    torch.cuda.synchronize()
    assert int(att.dev_status.item()) == 0
    return out, lse


# one tile a CTA; whole tiles; tiles in many ranges; in two or three
@pytest.mark.parametrize("lens_q,lens_k,at", [([600], [600], 400), ([4000], [4000], 1777), ([20], [4000], 2500),
                                              ([300, 20], [9000, 50], 8500)])
@pytest.mark.parametrize("power", [40, 47.3, 60, 115, 140])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("with_lse", [False, True])
def test_a_dominant_key_gives_its_value_exactly(sa, with_lse, d, power, lens_q, lens_k, at):  # noqa: F811
    # Key `at` scores `power` (base 2, to bf16) for every query, the others about 0 (a thousandth of the values' spread
    # of 2 is far): their weights are below 9000 * 2^-32 of the row, the sums, the division and its factor round by
    # 2^-21, so that the output is the value to 2^-18, and the value is a bf16 number.
    q, k, v, cq, ck = tp.inputs(90, lens_q, lens_k, 4, 2, d, device="cuda")
    q[..., 0] = 8.0 * math.sqrt(d / 64)
    k[..., 0] = 0.0
    k[at] = 0.0
    k[at, :, 0] = power * 0.6931471805599453
    # (values of one size, so that 2^-18 of the spread is far below a step of any)
    v = torch.where(v < 0, -1.0, 1.0).bfloat16() * (1 + torch.rand_like(v.float())).bfloat16()
    out, lse = run(sa, q, k, v, cq, ck, with_lse)
    n, m = lens_q[0], lens_k[0]
    first = max(0, at - (m - n))
    assert (out[first:n] == v[at].repeat_interleave(2, 0)).all()
    if with_lse:
        ref = (q[first:n, :, 0].double() * k[at, 0, 0].double()) / math.sqrt(d)
        assert ((lse[first:n].double() - ref).abs() <= 2.0 ** -17 + 2.0 ** -22 * ref.abs()).all()


@pytest.mark.parametrize("lens_q,lens_k", LENS)
@pytest.mark.parametrize("a", [240.0, 255.0, 1000.0])
def test_weights_that_are_all_the_same(sa, a, lens_q, lens_k):  # noqa: F811
    # each is 2 to the rounding of the reference, the same for all keys of a row
    q, k, v, cq, ck = tp.inputs(91, lens_q, lens_k, 4, 2, 64, device="cuda")
    q.fill_(a)
    k.fill_(a)
    out, lse = run(sa, q, k, v, cq, ck, True)
    check(out, lse, v, lens_q, lens_k, 64 * a * a / math.sqrt(64))
    assert torch.equal(run(sa, q, k, v, cq, ck, False)[0], out)
