"""Helpers of the packed attention tests: random packed sequences, a fast form
of the oracle and derived tolerances.

Tolerances.  With E = A (d + 8) 2^-23, A the largest sum |q k| scale over the
row's keys, a score is off by at most E, and an unnormalised weight, relative to
the row's reference, by 2 E + 2^-20 (the exponential).  It then rounds to bf16:
2^-8.  The output divides by the sum of the weights before or after that
rounding, so with e = 2 E + 2^-20 + n 2^-23 (n keys' fp32 sums) + 2^-8 the
weighted mean is off by at most e (sum p |v| + |o|) (1 + 2 e), plus half a step
of bf16 of the value, 2^-8.  The log-sum-exp adds unrounded weights: E + 2^-20 + n 2^-23 + 2^-22 |lse|.
A tile cut in r ranges rounds m + log2 l of each (|m| <= 2 (A + 10)): 2^-22 (A +
10) more, relative, and r more sums.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import packed as op


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def inputs(seed, lens_q, lens_k, hq, hkv, d, pad=0, sharp=1.0, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(lens_q) + pad, sum(lens_k) + pad
    q = (torch.randn(tq, hq, d, generator=g) * sharp).bfloat16()
    k = torch.randn(tk, hkv, d, generator=g).bfloat16()
    v = torch.randn(tk, hkv, d, generator=g).bfloat16()
    return q.to(device), k.to(device), v.to(device), cu_of(lens_q).to(device), cu_of(lens_k).to(device)


def reference(q, k, v, cu_q, cu_k, scale=None):
    """What oracle.packed.attend returns, in fp64 by whole sequences (CPU or GPU
    tensors; the results are CPU arrays)."""
    q, k, v = (t.double() for t in (q, k, v))
    cq, ck = cu_q.tolist(), cu_k.tolist()
    tq, hq, d = q.shape
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.full((tq, hq, d), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((tq, hq), float("nan"), dtype=torch.float64, device=q.device)
    absv, absqk = torch.zeros_like(o), torch.zeros_like(lse)
    for s in range(len(cq) - 1):
        n, m = cq[s + 1] - cq[s], ck[s + 1] - ck[s]
        if n == 0:
            continue
        rows = slice(cq[s], cq[s + 1])
        seen = (torch.arange(m, device=q.device) <=
                torch.arange(n, device=q.device)[:, None] + m - n)
        for h in range(hq):
            qq = q[rows, h]
            kk, vv = (x[ck[s]:ck[s + 1], h // group] for x in (k, v))
            x = torch.where(seen, qq @ kk.T * scale, -float("inf"))
            lse[rows, h] = torch.logsumexp(x, 1) if m else -float("inf")
            p = torch.where(seen, torch.exp(x - lse[rows, h][:, None]), 0.0)
            o[rows, h] = p @ vv
            absv[rows, h] = p @ vv.abs()
            a = torch.where(seen, qq.abs() @ kk.abs().T * scale, 0.0)
            absqk[rows, h] = a.amax(1) if m else 0.0
    return tuple(t.cpu().numpy() for t in (o, lse, absv, absqk))


def check(ref, out, lse, lens_q, lens_k, d):
    o, l, absv, absqk = ref
    rows = sum(lens_q)
    n = np.concatenate([np.maximum(0, np.arange(a) + b - a + 1) for a, b in zip(lens_q, lens_k)] or
                       [np.zeros(0)]).astype(np.float64)[:, None]
    E = absqk[:rows] * (d + 8) * 2.0 ** -23
    more = 2.0 ** -22 * (absqk[:rows] + 10) + 304 * 2.0 ** -23
    got = out.double().cpu().numpy()[:rows]
    o, absv = o[:rows], absv[:rows]
    e = (2 * E + 2.0 ** -20 + n * 2.0 ** -23 + more + 2.0 ** -8)[..., None]
    err = np.abs(got - o)
    tol = e * (absv + np.abs(o)) * (1 + 2 * e) + 2.0 ** -8 * np.maximum(np.abs(o), np.abs(got)) + 1e-30
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err / tol).max()
    if lse is not None:
        gl = lse.double().cpu().numpy()[:rows]
        none = np.broadcast_to(n == 0, gl.shape)
        assert (gl[none] == -np.inf).all()
        t = E + 2.0 ** -20 + n * 2.0 ** -23 + more + 2.0 ** -22 * np.abs(np.where(none, 0, l[:rows]))
        e = np.abs(gl[~none] - l[:rows][~none])
        assert (e <= t[~none]).all(), (e / t[~none]).max()
    if rows:
        assert (got[np.broadcast_to(n == 0, got.shape[:2])] == 0).all()


def same(got, ref):
    assert torch.equal(got.view(torch.int16) if got.dtype == torch.bfloat16 else got,
                       ref.view(torch.int16) if ref.dtype == torch.bfloat16 else ref)
