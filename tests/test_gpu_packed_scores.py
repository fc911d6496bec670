"""Packed causal attention of scores too large for their logarithm's rounding.

Queries and keys of one value a give every score d a^2 scale, exactly: 64 products
of integers below 2^8 times a power of two.  So every weight is the same, a row's
output is the mean of the values that it sees, and the only roundings are those of
sums (n 2^-23 of the values' mean size), of the division (2^-22) and of the output
(2^-8 of it); log-sum-exps round to 2^-22 of themselves."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import _packed as tp  # noqa: E402
from tests.test_gpu_packed import run, sa  # noqa: E402, F401

pytestmark = pytest.mark.gpu

# one tile a CTA; whole tiles; tiles in many ranges; in two or three
LENS = [([60], [60]), ([700, 40], [700, 40]), ([20, 5], [4000, 300]), ([100] * 50, [2000] * 50)]


def means(v, lens_q, lens_k):
    """Mean value, and size, of what every query sees, and how many keys these are."""
    o, size, n, at = [], [], [], 0
    for a, b in zip(lens_q, lens_k):
        x = v[at:at + b].double()
        seen = torch.arange(1, b + 1, device=v.device, dtype=torch.float64)[:, None, None]
        o.append((x.cumsum(0) / seen)[b - a:])
        size.append((x.abs().cumsum(0) / seen)[b - a:])
        n.append(seen[b - a:])
        at += b
    return torch.cat(o), torch.cat(size), torch.cat(n)


def check(out, lse, v, lens_q, lens_k, score):
    o, size, n = means(v, lens_q, lens_k)
    group = out.shape[1] // v.shape[1]
    o, size = (t.repeat_interleave(group, 1) for t in (o, size))
    assert torch.isfinite(out).all()
    err = (out.double() - o).abs()
    assert (err <= (n * 2.0 ** -23 + 2.0 ** -22) * (size + o.abs()) + 2.0 ** -8 * o.abs()).all()
    ref = score + n[..., 0].log()
    assert ((lse.double() - ref).abs() <= 2.0 ** -22 * ref.abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("lens_q,lens_k", LENS)
@pytest.mark.parametrize("a,b", [(30720.0, 30720.0), (40960.0, 40960.0), (30720.0, -30720.0), (40960.0, -40960.0),
                                 (2.0 ** 50, 2.0 ** 50)])
def test_every_score_the_same(sa, a, b, lens_q, lens_k):  # noqa: F811
    q, k, v, cq, ck = tp.inputs(80, lens_q, lens_k, 4, 2, 64, device="cuda")
    q.fill_(a)
    k.fill_(b)
    out, lse = run(sa, 4, 2, 64, q, k, v, cq, ck)
    check(out, lse, v, lens_q, lens_k, 64 * a * b / math.sqrt(64))


@pytest.mark.parametrize("lens_q,lens_k", LENS)
def test_every_score_the_same_and_sums_of_values_out_of_range(sa, lens_q, lens_k):  # noqa: F811
    # the mean of the values is in range, their sum is not
    q, k, v, cq, ck = tp.inputs(81, lens_q, lens_k, 4, 2, 128, device="cuda")
    q.fill_(30720.0)
    k.fill_(30720.0)
    v = (v.float().abs() * 1.0e38).clamp(max=3.3e38).bfloat16()
    v[::3] = -v[::3]
    v[:40] = v[:40].abs()
    out, lse = run(sa, 4, 2, 128, q, k, v, cq, ck)
    check(out, lse, v, lens_q, lens_k, 128 * 30720.0 ** 2 / math.sqrt(128))


@pytest.mark.parametrize("lens_q,lens_k,at", [([60], [60], 33), ([700], [700], 400), ([20], [4000], 2500)])
def test_one_key_above_the_others(sa, lens_q, lens_k, at):  # noqa: F811
    # a bf16 step more is 2^-7 of the score: the queries that see it get its value alone
    q, k, v, cq, ck = tp.inputs(82, lens_q, lens_k, 2, 1, 64, device="cuda")
    q.fill_(30720.0)
    k.fill_(30720.0)
    k[at] = 30848.0
    out, lse = run(sa, 2, 1, 64, q, k, v, cq, ck)
    first = max(0, at - (lens_k[0] - lens_q[0]))
    assert (out[first:] == v[at]).all()
    ref = 64 * 30720.0 * 30848.0 / 8
    assert ((lse[first:].double() - ref).abs() <= 2.0 ** -22 * ref).all()
    check(out[:first], lse[:first], v, [first], [at] if first else [0], 64 * 30720.0 ** 2 / 8)


@pytest.mark.parametrize("lens_q,lens_k,low", [([60], [60], 40), ([700], [700], 400), ([20], [4000], 1500),
                                               ([20], [4000], 3990), ([100] * 50, [2000] * 50, 1100)])
@pytest.mark.parametrize("by", ["infinity", "overflow"])
def test_keys_whose_scores_are_minus_infinity(sa, by, lens_q, lens_k, low):  # noqa: F811
    # They weigh nothing beside others, whole blocks and ranges of them too; a row that sees no other key has no mean
    d = 64
    q, k, v, cq, ck = tp.inputs(83, lens_q, lens_k, 4, 2, d, device="cuda")
    q[..., 0] = 1.0 if by == "infinity" else 1e20
    k[..., 0] = 0.0
    at = [(sum(lens_k[:i]), n, m) for i, (n, m) in enumerate(zip(lens_q, lens_k))]
    for first, _, _ in at:
        k[first:first + low] = 0.0
        k[first:first + low, :, 0] = -math.inf if by == "infinity" else -1e20
    out, lse = run(sa, 4, 2, d, q, k, v, cq, ck)
    # the same queries behind the other keys alone
    keep = torch.cat([torch.arange(first + low, first + m) for first, _, m in at]).cuda()
    rest = [m - low for m in lens_k]
    ref = tp.reference(q, k[keep], v[keep], cq, tp.cu_of(rest).cuda())
    sees = torch.cat([torch.arange(m - n, m) >= low for _, n, m in at])
    assert out[~sees.cuda()].isnan().all() and (lse[~sees.cuda()] == -math.inf).all()
    got, gl = out.clone(), lse.clone()
    got[~sees.cuda()], gl[~sees.cuda()] = 0.0, -math.inf
    tp.check(ref, got, gl, lens_q, rest, d)
