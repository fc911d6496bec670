"""Oracle: pages and slots of new tokens, with lists (test infrastructure only;
see the package docstring)."""
from __future__ import annotations

import numpy as np


def grow(table, lens, owned, free, page, spans, counts=None, ended=None, start=None, tokens=None,
         weights=None, positions=None):
    """table [B, H, max_pages], lens and owned [B, H], free: the list of free
    pages; spans: (first, end) of each sequence's tokens.  Returns a dict of the
    new state (arrays of the same shapes, `free` a list) and of slots [H,
    tokens], token_positions, granted and start."""
    table, lens, owned = table.copy(), lens.copy(), owned.copy()
    B, H, max_pages = table.shape
    ended = [False] * B if ended is None else ended
    weights = None if weights is None else weights.copy()
    positions = None if positions is None else positions.copy()
    slots = np.full((H, tokens), -1, np.int64)
    token_positions = np.zeros(tokens, np.int64)
    granted, first = np.zeros(B, np.int64), np.zeros(B, np.int64)
    want = np.zeros(B, np.int64)
    stack = list(free)
    for b in range(B):
        if ended[b]:
            lens[b] = 0
        want[b] = spans[b][1] - spans[b][0] if counts is None else counts[b]
        if want[b] > max_pages * page - lens[b].max():
            want[b] = 0
        first[b] = (0 if ended[b] else start[b]) if start is not None else lens[b].max()
    need = -(-(lens + want[:, None]) // page)
    for b in range(B):
        for g in range(H):
            if owned[b, g] > need[b, g]:
                stack += table[b, g, need[b, g]:owned[b, g]].tolist()
                owned[b, g] = need[b, g]
    room, asked = len(stack), 0
    for b in range(B):
        more = int(np.maximum(need[b] - owned[b], 0).sum())
        asked += more
        if more and asked > room:
            continue
        granted[b] = want[b]
        for g in range(H):
            while owned[b, g] < need[b, g]:
                table[b, g, owned[b, g]] = stack.pop()
                owned[b, g] += 1
            for i in range(int(want[b])):
                at = int(lens[b, g]) + i
                slots[g, spans[b][0] + i] = int(table[b, g, at // page]) * page + at % page
                token_positions[spans[b][0] + i] = first[b] + i
                if weights is not None:
                    weights[b, g, at] = 0
                if positions is not None:
                    positions[b, g, at] = first[b] + i
        lens[b] += granted[b]
    return {"table": table, "lens": lens, "owned": owned, "free": stack, "slots": slots,
            "token_positions": token_positions, "granted": granted, "start": first + granted,
            "weights": weights, "positions": positions}
