"""Oracle: causal attention of packed sequences, in fp64 (test infrastructure
only; see the package docstring)."""
from __future__ import annotations

import math

import numpy as np


def attend(q, k, v, cu_q, cu_k, scale=None):
    """q [Tq, Hq, d]; k, v [Tk, Hkv, d]; cu_q, cu_k [B + 1].  Query i of a
    sequence of n queries and m keys sees its keys u <= i + m - n.  Returns o
    (0 for a query that sees none), lse (-infinity there) and two bounds that a
    test of rounding needs: the sum over keys of p |v|, and the largest sum
    over elements of |q k| scale.  Rows in no sequence are NaN."""
    Tq, Hq, d = q.shape
    group = Hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = np.full((Tq, Hq, d), np.nan)
    lse = np.full((Tq, Hq), np.nan)
    absv, absqk = np.zeros((Tq, Hq, d)), np.zeros((Tq, Hq))
    for q0, q1, k0, k1 in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        n, m = int(q1) - int(q0), int(k1) - int(k0)
        for i in range(n):
            seen = max(0, i + m - n + 1)
            t = int(q0) + i
            for h in range(Hq):
                if seen == 0:
                    o[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                kk = k[k0:k0 + seen, h // group].astype(np.float64)
                vv = v[k0:k0 + seen, h // group].astype(np.float64)
                qq = q[t, h].astype(np.float64)
                s = kk @ qq * scale
                top = s.max()
                w = np.exp(s - top)
                total = w.sum()
                p = w / total
                o[t, h], lse[t, h] = p @ vv, top + math.log(total)
                absv[t, h] = p @ np.abs(vv)
                absqk[t, h] = (np.abs(kk) @ np.abs(qq)).max() * scale
    return o, lse, absv, absqk
