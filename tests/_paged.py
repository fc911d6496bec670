"""Helpers of the paged cache tests: random caches and derived tolerances.

Tolerances.  With E = A (d + 8) 2^-23, A the largest sum |q k| / sqrt(d) over
the row's tokens, a score (a sum of d fp32 products, scaled) is off by at most
E.  A probability is exp(s - lse): both terms are off by at most E, the
exponential and the sums add 2^-20 + n 2^-23 for n tokens, and the split of an
unnormalised weight into two bf16 parts leaves at most (2^-8)^2 of it.  So
  |do|      <= (2 E + 2^-16 + 2^-20 + n 2^-23) sum p |v|, plus half a step of
               the output type (bf16 2^-8, fp32 2^-24) of the value;
  |dlse|    <= E + 2^-20 + n 2^-23 + 2^-22 |lse|;
  |dweight| <= (2 E + 2^-20 + n 2^-23) G (probabilities are at most 1 each: the
               bound is relative to the sum of the row's probabilities), plus
               2^-22 of the sum (additions and the final rounding).
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged as op


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(x, dtype=torch.float32).bfloat16()


def random_cache(seed, lens, hkv, d, page, max_pages=None, spare=3, weights=True, interleaved=False,
                 junk=True):
    """CPU tensors of a cache: rows' pages in random order, table entries behind
    a row's last page -1, NaN / infinity / huge values in every unused slot."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.as_tensor(lens, dtype=torch.int32)
    if lens.dim() == 1:
        lens = lens[:, None].expand(-1, hkv).contiguous()
    b = lens.shape[0]
    need = (lens.long() + page - 1) // page
    mp = int(max(1, need.max())) if max_pages is None else max_pages
    total = int(need.sum()) + spare
    shape = (total, 2, page, d) if interleaved else (2, total, page, d)
    both = torch.randn(shape, generator=g).bfloat16()
    k, v = (both[:, 0], both[:, 1]) if interleaved else (both[0], both[1])
    perm = torch.randperm(total, generator=g).int()
    table = torch.full((b, hkv, mp), -1, dtype=torch.int32)
    used = torch.zeros(total, page, dtype=torch.bool)
    at = 0
    for x in range(b):
        for h in range(hkv):
            n = int(need[x, h])
            table[x, h, :n] = perm[at:at + n]
            at += n
            t = torch.arange(int(lens[x, h]))
            used[table[x, h].long()[t // page], t % page] = True
    if junk:
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])
        pick = bad[torch.randint(0, 4, (total, page, 1), generator=g)].bfloat16()
        for t in (k, v):
            t.copy_(torch.where(used[..., None], t, pick))
    w = torch.rand(b, hkv, mp * page, generator=g) if weights else None
    pos = torch.arange(mp * page, dtype=torch.int32).expand(b, hkv, -1).contiguous()
    return {"k": k, "v": v, "table": table, "lens": lens, "weights": w, "positions": pos,
            "page": page}


def to_gpu(c, sa, with_weights=True, **kw):
    """The cache's tensors on the GPU (pool views keep their strides) and a PagedCache."""
    dev = {}
    base = c["k"]._base if c["k"]._base is not None else None
    if base is not None:
        gb = base.cuda()
        inter = c["k"].stride(0) != c["k"].shape[1] * c["k"].shape[2]
        dev["k"], dev["v"] = (gb[:, 0], gb[:, 1]) if inter else (gb[0], gb[1])
    else:
        dev["k"], dev["v"] = c["k"].cuda(), c["v"].cuda()
    for n in ("table", "lens", "weights", "positions"):
        dev[n] = c[n].cuda() if c[n] is not None else None
    cache = sa.PagedCache(dev["k"], dev["v"], dev["table"], dev["lens"],
                          weights=dev["weights"] if with_weights else None,
                          positions=dev["positions"], **kw)
    return dev, cache


def f64(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def slot_mask(table, lens, page, pages):
    """Which (page, row) of the pool the rows' slots are."""
    used = np.zeros((pages, page), dtype=bool)
    for b in range(lens.shape[0]):
        for g in range(lens.shape[1]):
            t = np.arange(int(lens[b, g]))
            used[table[b, g].numpy()[t // page], t % page] = True
    return used


def check_attend(c, q, out, lse, weights_out=None, weights_before=None, d=None):
    """Outputs (CPU or GPU tensors) against the oracle at the derived bounds."""
    page = c["page"]
    G = q.shape[1] // c["lens"].shape[1]
    wb = c["weights"] if weights_before is None else weights_before
    o, l, w, absv, absqk = op.attend(f64(q), f64(c["k"]), f64(c["v"]), f64(c["table"]),
                                     f64(c["lens"]),
                                     None if weights_out is None else f64(wb))
    d = q.shape[2]
    n = np.repeat(f64(c["lens"]), G, axis=1).astype(np.float64)       # [Bt, Hq]
    E = absqk * (d + 8) * 2.0 ** -23
    rel = 2 * E + 2.0 ** -16 + 2.0 ** -20 + n * 2.0 ** -23
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    got = f64(out)
    err = np.abs(got - o)
    tol = rel[..., None] * absv + half * np.maximum(np.abs(o), np.abs(got)) + 1e-30
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err / tol).max()
    if lse is not None:
        gl = f64(lse)
        empty = n == 0
        assert (gl[empty] == -np.inf).all()
        e = np.abs(gl[~empty] - l[~empty])
        t = (E + 2.0 ** -20 + n * 2.0 ** -23)[~empty] + 2.0 ** -22 * np.abs(l[~empty])
        assert (e <= t).all(), (e / t).max()
    if weights_out is not None:
        gw = f64(weights_out)
        Bt, Hkv = c["lens"].shape
        for b in range(Bt):
            for g in range(Hkv):
                m = int(c["lens"][b, g])
                if m == 0:
                    continue
                Em = E[b, g * G:(g + 1) * G].max()
                add = w[b, g, :m] - f64(wb)[b, g, :m]
                t = (2 * Em + 2.0 ** -20 + m * 2.0 ** -23) * add + 2.0 ** -22 * np.abs(w[b, g, :m])
                e = np.abs(gw[b, g, :m] - w[b, g, :m])
                assert (e <= t).all(), (e / t).max()
