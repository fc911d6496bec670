"""Oracle: a paged key-value cache with a length per (sequence, KV head), in
fp64 (test infrastructure only; see the package docstring).

Pools k_pages, v_pages [num_pages, page, d]; table [Bt, Hkv, max_pages]; lens
[Bt, Hkv]; weights, positions [Bt, Hkv, max_pages * page].  The functions
return new arrays and leave their inputs alone.
"""
from __future__ import annotations

import math

import numpy as np


def slot_rows(table_row: np.ndarray, slots: np.ndarray, page: int):
    """(page number, row in the page) of the given slots of one cache row."""
    return table_row[slots // page], slots % page


def append(k_pages, v_pages, table, lens, k_new, v_new, counts, start, weights, positions):
    """k_new, v_new [Bt, Hkv, T, d]; counts, start [Bt]."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    lens, weights, positions = lens.copy(), weights.copy(), positions.copy()
    page = k_pages.shape[1]
    Bt, Hkv = lens.shape
    for b in range(Bt):
        for g in range(Hkv):
            n, m = int(lens[b, g]), int(counts[b])
            slots = np.arange(n, n + m)
            p, x = slot_rows(table[b, g], slots, page)
            k_pages[p, x] = k_new[b, g, :m]
            v_pages[p, x] = v_new[b, g, :m]
            weights[b, g, n:n + m] = 0
            positions[b, g, n:n + m] = start[b] + np.arange(m)
            lens[b, g] = n + m
    return k_pages, v_pages, lens, weights, positions


def attend(q, k_pages, v_pages, table, lens, weights=None):
    """o [Bt, Hq, d], lse [Bt, Hq], weights plus the summed probabilities, and
    two bounds a test of rounding needs, per query head: the sum over tokens of
    p |v| (per element) and the largest sum over elements of |q k| / sqrt(d)."""
    Bt, Hq, d = q.shape
    Hkv = lens.shape[1]
    page, group = k_pages.shape[1], Hq // Hkv
    o = np.zeros((Bt, Hq, d))
    lse = np.full((Bt, Hq), -np.inf)
    absv = np.zeros((Bt, Hq, d))
    absqk = np.zeros((Bt, Hq))
    out_w = None if weights is None else weights.astype(np.float64)
    for b in range(Bt):
        for g in range(Hkv):
            n = int(lens[b, g])
            if n == 0:
                continue
            p, x = slot_rows(table[b, g], np.arange(n), page)
            k, v = k_pages[p, x].astype(np.float64), v_pages[p, x].astype(np.float64)
            for h in range(g * group, (g + 1) * group):
                qh = q[b, h].astype(np.float64)
                s = k @ qh / math.sqrt(d)
                top = s.max()
                e = np.exp(s - top)
                lse[b, h] = top + math.log(e.sum())
                prob = e / e.sum()
                o[b, h] = prob @ v
                absv[b, h] = prob @ np.abs(v)
                absqk[b, h] = (np.abs(k) @ np.abs(qh)).max() / math.sqrt(d)
                if out_w is not None:
                    out_w[b, g, :n] += prob
    return o, lse, out_w, absv, absqk


def kept_slots(weights, positions, keep: int, sinks: int, recent: int):
    """The slots one row keeps, ascending."""
    n = len(weights)
    newest = int(positions.max()) if n else 0
    order = []
    for t in range(n):
        forced = positions[t] < sinks or positions[t] > newest - recent
        w = float(weights[t])
        order.append((0 if forced else 1, 0.0 if forced else (math.inf if math.isnan(w) else -w),
                      0 if forced or not math.isnan(w) else 1, t))
    order.sort()
    return sorted(x[3] for x in order[:keep])


def evict(k_pages, v_pages, table, lens, weights, positions, keep, sinks, recent):
    """Cuts each row to keep[g] tokens; kept tokens behind the new length move,
    lowest first, into the evicted slots before it, lowest first."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    lens, weights, positions = lens.copy(), weights.copy(), positions.copy()
    page = k_pages.shape[1]
    Bt, Hkv = lens.shape
    for b in range(Bt):
        for g in range(Hkv):
            n = int(lens[b, g])
            m = min(n, int(keep[g]))
            if n <= m:
                continue
            kept = kept_slots(weights[b, g, :n], positions[b, g, :n], m, sinks, recent)
            have = set(kept)
            dst = np.array([t for t in range(m) if t not in have], dtype=np.int64)
            src = np.array([t for t in kept if t >= m], dtype=np.int64)
            sp, sx = slot_rows(table[b, g], src, page)
            dp, dx = slot_rows(table[b, g], dst, page)
            k_pages[dp, dx] = k_pages[sp, sx]
            v_pages[dp, dx] = v_pages[sp, sx]
            weights[b, g, dst] = weights[b, g, src]
            positions[b, g, dst] = positions[b, g, src]
            lens[b, g] = m
    return k_pages, v_pages, lens, weights, positions
