"""Cases of the paged key-value cache operators, with their plain forms.

The cache holds, for every (sequence, KV head) row, `lens[b, g]` tokens in pages of `page` tokens; `table[b, g]` lists the
row's pages, so each head may keep its own number of tokens.  Three operators work on it:

  append   writes new tokens' keys and values behind each row's last token (weight 0, their positions beside them);
  attend   softmax attention of one new token's query heads over each row's tokens, its log-sum-exp, and (where the cache
           keeps weights) adds every token's attention probability, summed over the row's query heads, to the token's weight;
  evict    keeps `keep[g]` tokens of each row: the first `sinks` positions, the last `recent` ones and then those of the
           largest weight; kept tokens behind the new length move, in order, into the slots of evicted ones before it.

Page 0 is a null page: it belongs to no row, and a row's table names it behind the row's last page.
"""
import math

import torch

own = False

PAGES = (16, 32, 64, 128, 256)
HEADS = ((8, 2, 64), (16, 16, 64), (32, 8, 128), (28, 4, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128))


def _attend(name, batch, hq, hkv, d, page, lo, hi, per_head=False, weights=False, f32=False):
    return {"name": name, "op": "attend", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "page": page, "lo": lo, "hi": hi,
            "per_head": per_head, "weights": weights, "f32": f32}


def _append(name, batch, hq, hkv, d, page, lo, hi, new, ragged=False, fused=False):
    return {"name": name, "op": "append", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "page": page, "lo": lo, "hi": hi,
            "new": new, "ragged": ragged, "fused": fused}


def _evict(name, batch, hkv, d, page, lo, hi, keep_lo, keep_hi, extra=0):
    return {"name": name, "op": "evict", "batch": batch, "hkv": hkv, "d": d, "page": page, "lo": lo, "hi": hi,
            "keep_lo": keep_lo, "keep_hi": keep_hi, "extra": extra}


def listed():
    return [
        # one user's chat, a short context: latency
        _attend("attend_chat", 1, 32, 8, 128, 16, 700, 700),
        # a batch of conversations of any length
        _attend("attend_batch", 32, 32, 8, 128, 16, 0, 8192),
        # the decode workload's shape: 16 sequences of 64K tokens, 7 query heads a KV head
        _attend("attend_long", 16, 28, 4, 128, 32, 65536, 65536),
        # one sequence at the longest prefill's length, odd: all processors on few rows
        _attend("attend_one_128k", 1, 64, 8, 128, 64, 131071, 131071),
        # the small model's heads, d = 64, many sequences
        _attend("attend_d64", 64, 8, 2, 64, 16, 1, 4096),
        # heads that keep different numbers of tokens after evictions, and go on accumulating weights
        _attend("attend_weights", 16, 32, 8, 128, 32, 512, 8192, per_head=True, weights=True),
        # a decode step's tokens, as views of the fused projection's output
        _append("append_step", 64, 32, 8, 128, 16, 1, 8000, 1, fused=True),
        # a prompt's keys and values as the prefill layer takes them, an odd length
        _append("append_prompt", 1, 32, 8, 128, 64, 0, 0, 32767),
        # chunks of prompts behind what is there, of differing lengths, some of them empty
        _append("append_chunk", 16, 28, 4, 128, 32, 1, 4096, 1024, ragged=True, fused=True),
        # a decode step's eviction: each row is a page over its budget
        _evict("evict_step", 32, 8, 128, 32, 0, 0, 512, 2048, extra=32),
        # after a prompt: per-head budgets from a 32nd to a quarter
        _evict("evict_prompt", 4, 8, 128, 64, 32768, 32768, 1024, 8192),
        # the small model's 4K sequences
        _evict("evict_d64", 8, 2, 64, 16, 2048, 4096, 512, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "evict"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice(PAGES)
    batch = _log(rng, 1, 64)
    rows = batch * hkv
    if op == "attend":
        hi = _log(rng, 1, max(2, min(131072, (1 << 29) // (rows * d))))  # at most 2 GiB of keys and values
        lo = hi if rng.random() < 0.4 else rng.randint(0, hi)
        c = _attend("", batch, hq, hkv, d, page, lo, hi, rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.2)
    elif op == "append":
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(4, min(32768, (1 << 26) // (rows * d))))
        hi = _log(rng, 1, max(2, min(16384, (1 << 26) // (rows * d))))
        c = _append("", batch, hq, hkv, d, page, rng.randint(0, hi), hi, new, rng.random() < 0.5, rng.random() < 0.5)
    else:
        hi = _log(rng, 64, max(128, min(65536, (1 << 27) // (rows * d))))
        keep_hi = _log(rng, 32, hi)
        extra = rng.randint(1, 64) if rng.random() < 0.4 else 0
        c = _evict("", batch, hkv, d, page, rng.randint(max(1, hi // 2), hi), hi, rng.randint(max(24, keep_hi // 4), keep_hi),
                   keep_hi, extra)
    del c["name"]
    return c


SINKS, RECENT = 4, 16


def _keep(c):
    n = c["hkv"]
    return [int(round(c["keep_lo"] * (c["keep_hi"] / c["keep_lo"]) ** (g / max(1, n - 1)))) for g in range(n)]


def _tokens(c):
    """The most tokens a row of this case holds."""
    if c["op"] == "append":
        return c["hi"] + c["new"]
    return c["keep_hi"] + c["extra"] if c["op"] == "evict" and c["extra"] else c["hi"]


def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    opt = {"device": "cuda", "generator": g}
    b, h, d, page = c["batch"], c["hkv"], c["d"], c["page"]
    rows, cap_pages = b * h, -(-_tokens(c) // page)
    s = {}
    if c["op"] == "evict" and c["extra"]:
        s["lens"] = (torch.tensor(_keep(c), device="cuda") + c["extra"]).expand(b, h).int().contiguous()
    elif c.get("per_head"):
        s["lens"] = torch.randint(c["lo"], c["hi"] + 1, (b, h), dtype=torch.int32, **opt)
    else:
        s["lens"] = torch.randint(c["lo"], c["hi"] + 1, (b, 1), dtype=torch.int32, **opt).expand(b, h).contiguous()
    # every row's pages, drawn from a pool in random order; page 0 stays the null page
    pages = torch.randperm(rows * cap_pages, **opt).view(b, h, cap_pages).int() + 1
    need = s["lens"] + (c["new"] if c["op"] == "append" else 0)
    used = torch.arange(cap_pages, device="cuda") * page < need[..., None]
    s["table"] = torch.where(used, pages, 0).int().contiguous()
    pool = (rows * cap_pages + 1, page, d)
    s["k_pages"] = torch.randn(pool, dtype=torch.bfloat16, **opt)
    s["v_pages"] = torch.randn(pool, dtype=torch.bfloat16, **opt)
    if c["op"] == "attend":
        # heads of differing sharpness, as the prefill and decode inputs have
        sharp = torch.exp(torch.rand(c["hq"], 1, **opt) * 1.4 - 0.7)
        s["q"] = (torch.randn(b, c["hq"], d, **opt) * sharp).bfloat16()
        s["o"] = torch.zeros(b, c["hq"], d, dtype=torch.float32 if c["f32"] else torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(b, c["hq"], device="cuda")
    if c["op"] == "evict" or c.get("weights"):
        s["weights"] = torch.exp(2 * torch.randn(b, h, cap_pages * page, **opt) - 4)
        s["weights_out"] = torch.zeros_like(s["weights"])
    if c["op"] == "append":
        n, hq = c["new"], c["hq"]
        if c["fused"]:
            qkv = torch.randn(b, n, hq + 2 * h, d, dtype=torch.bfloat16, **opt)
            s["k"], s["v"] = qkv[:, :, hq:hq + h].transpose(1, 2), qkv[:, :, hq + h:].transpose(1, 2)
        else:
            s["k"] = torch.randn(b, h, n, d, dtype=torch.bfloat16, **opt)
            s["v"] = torch.randn(b, h, n, d, dtype=torch.bfloat16, **opt)
        s["counts"] = torch.randint(0, n + 1, (b,), dtype=torch.int32, **opt) if c["ragged"] else \
            torch.full((b,), n, dtype=torch.int32, device="cuda")
        s["start"] = s["lens"].amax(1) + torch.randint(0, 1000, (b,), dtype=torch.int32, **opt)
        s["weights"] = torch.rand(b, h, cap_pages * page, **opt)
        s["positions"] = torch.arange(cap_pages * page, dtype=torch.int32, device="cuda").expand(b, h, -1).contiguous()
        s["lens_out"] = torch.zeros_like(s["lens"])
    if c["op"] == "evict":
        # positions seen so far: increasing, with gaps, and out of order in the slots that earlier evictions refilled
        cap = cap_pages * page
        pos = (torch.randint(1, 4, (b, h, cap), **opt) if c["extra"] else torch.ones(b, h, cap, device="cuda").long()).cumsum(-1) - 1
        if c["extra"]:
            at = torch.rand(b, h, cap, **opt)
            slot = torch.arange(cap, device="cuda")
            at = torch.where(slot < s["lens"][..., None] - c["extra"], at, 1.0 + slot)
            pos = pos.gather(-1, at.argsort(-1))
        s["positions"] = pos.int().contiguous()
        s["positions_out"] = torch.zeros_like(s["positions"])
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["keep"] = _keep(c)
        s["keep_each"] = torch.tensor(s["keep"], device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import head_heterogeneous_block_gb300 as sa
        s["cache"] = sa.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["lens"], weights=s.get("weights"),
                                   positions=s.get("positions"), num_q_heads=case.get("hq"))
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attend(s):
    c, page, d = s["case"], s["case"]["page"], s["case"]["d"]
    b, hq, h = c["batch"], c["hq"], c["hkv"]
    cap = s["table"].shape[-1] * page
    at = s["table"].long()
    k = s["k_pages"][at].view(b, h, cap, d).float()
    v = s["v_pages"][at].view(b, h, cap, d).float()
    live = torch.arange(cap, device="cuda") < s["lens"][..., None]          # [b, h, cap]
    x = s["q"].float().view(b, h, hq // h, d) @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    x = torch.where(live[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p = torch.where(some, p / total, 0.0)
    v = torch.where(live[..., None], v, 0.0)
    s["o"].copy_((p @ v).view(b, hq, d))
    s["lse"].copy_((top + torch.log(total)).view(b, hq))
    out = {"o": s["o"], "lse": s["lse"]}
    if c["weights"]:
        s["weights_out"].copy_(torch.where(live, s["weights"] + p.sum(2), s["weights_out"]))
        out["weights"] = s["weights_out"]
    return out


def _flat(s, slot):
    """Row numbers, in the pools seen as [pages * page, d], of the given slots [b, h, n]."""
    page = s["case"]["page"]
    return s["table"].long().gather(-1, slot // page) * page + slot % page


def _plain_append(s):
    c, d = s["case"], s["case"]["d"]
    cap = s["table"].shape[-1] * c["page"]
    t = torch.arange(c["new"], device="cuda")
    slot = s["lens"].long()[..., None] + t
    new = t < s["counts"][:, None, None]
    row = torch.where(new, _flat(s, slot.clamp(max=cap - 1)), 0).flatten()  # what is not new goes to the null page
    for name, pool in (("k", s["k_pages"]), ("v", s["v_pages"])):
        null = pool[0].clone()
        pool.view(-1, d)[row] = s[name].reshape(-1, d)
        pool[0] = null
    behind = torch.arange(cap, device="cuda") - s["lens"].long()[..., None]
    fresh = (behind >= 0) & (behind < s["counts"][:, None, None])
    s["weights"].copy_(torch.where(fresh, 0.0, s["weights"]))
    s["positions"].copy_(torch.where(fresh, s["start"][:, None, None] + behind, s["positions"]))
    s["lens_out"].copy_(s["lens"] + s["counts"][:, None])
    return {"lens": s["lens_out"], "k": s["k_pages"], "v": s["v_pages"], "weights": s["weights"], "positions": s["positions"]}


def _plain_evict(s):
    d = s["case"]["d"]
    b, h, cap = s["weights"].shape
    n = s["lens"].long()[..., None]
    keep = s["keep_each"][:, None]
    short = torch.minimum(n, keep)                                           # the new lengths
    slot = torch.arange(cap, device="cuda").expand(b, h, cap)
    live = slot < n
    newest = torch.where(live, s["positions"], -1).amax(-1, keepdim=True)
    forced = (s["positions"] < SINKS) | (s["positions"] > newest - RECENT)
    key = torch.where(forced, math.inf, s["weights"])
    key = torch.where(live, key, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices               # ties: the lowest slot first
    rank = torch.empty_like(order).scatter_(-1, order, slot)
    kept = live & (rank < keep)
    hole = ~kept & (slot < short)
    source = torch.where(kept & (slot >= short), slot, cap).sort(-1).values  # in order, then cap
    nth = (hole.long().cumsum(-1) - 1).clamp(min=0)
    src = torch.where(hole, source.gather(-1, nth), slot)[..., :max(s["keep"])]
    dst = slot[..., :max(s["keep"])]
    ok = dst < short
    src = torch.where(ok, src, 0)
    to, at = torch.where(ok, _flat(s, dst), 0).flatten(), _flat(s, src).flatten()
    for pool in (s["k_pages"], s["v_pages"]):
        null = pool[0].clone()
        pool.view(-1, d)[to] = pool.view(-1, d)[at]
        pool[0] = null
    for name in ("weights", "positions"):
        part = s[name + "_out"][..., :dst.shape[-1]]
        part.copy_(torch.where(ok, s[name].gather(-1, src), part))
    s["lens_out"].copy_(short[..., 0])
    return {"lens": s["lens_out"], "k": s["k_pages"], "v": s["v_pages"], "weights": s["weights_out"],
            "positions": s["positions_out"]}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}[op](s)
    cache = s["cache"]
    if op == "attend":
        cache.attend(s["q"], out=s["o"], lse=s["lse"], weights_out=s.get("weights_out"))
        out = {"o": s["o"], "lse": s["lse"]}
        if s["case"]["weights"]:
            out["weights"] = s["weights_out"]
        return out
    if op == "append":
        cache.append(s["k"], s["v"], counts=s["counts"], start=s["start"], lens_out=s["lens_out"])
        return {"lens": s["lens_out"], "k": s["k_pages"], "v": s["v_pages"], "weights": s["weights"],
                "positions": s["positions"]}
    cache.evict(s["keep"], sinks=SINKS, recent=RECENT, lens_out=s["lens_out"], weights_out=s["weights_out"],
                positions_out=s["positions_out"])
    return {"lens": s["lens_out"], "k": s["k_pages"], "v": s["v_pages"], "weights": s["weights_out"],
            "positions": s["positions_out"]}


def work(case):
    c = case
    rows, d = c["batch"] * c["hkv"], c["d"]
    mean = (c["lo"] + c["hi"]) / 2
    if c["op"] == "attend":
        tokens = rows * mean
        heads = c["batch"] * c["hq"]
        return {"bytes": tokens * 4 * d + heads * (2 * d + (4 if c["f32"] else 2) * d + 4) + tokens / c["page"] * 4 + rows * 4
                + (tokens * 8 if c["weights"] else 0),
                "flops": tokens * (c["hq"] // c["hkv"]) * 4 * d}
    if c["op"] == "append":
        tokens = rows * c["new"] * (0.5 if c["ragged"] else 1)
        return {"bytes": tokens * (8 * d + 8) + tokens / c["page"] * 4 + rows * 8 + c["batch"] * 8, "flops": 0}
    total = moved = kept = 0.0
    for k in _keep(c):
        n = k + c["extra"] if c["extra"] else mean
        k = min(n, k)
        total, kept = total + n, kept + k
        # kept tokens lie evenly over the row, but for the last ones, which stay: those behind the new length move
        moved += min(n - k, RECENT + (k - RECENT) * (n - k) / n)
    return {"bytes": c["batch"] * (total * 8 + kept * 8 + moved * 8 * d + c["hkv"] * 8), "flops": c["batch"] * total}


# ---------------------------------------------------------------- in 64 bits
def _row_tokens(c, s, b, h, slots):
    """Pool row numbers of the slots of one row of the cache."""
    page = c["page"]
    return s["table"][b, h].long()[slots // page] * page + slots % page


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    d = c["d"]
    kf, vf = s["k_pages"].view(-1, d), s["v_pages"].view(-1, d)
    if c["op"] == "attend":
        group = c["hq"] // c["hkv"]
        o = torch.zeros(c["batch"], c["hq"], d, dtype=torch.float64, device="cuda")
        lse = torch.full((c["batch"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
        w = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda") if c["weights"] else None
        lens = s["lens"].tolist()
        for b in range(c["batch"]):
            for h in range(c["hkv"]):
                n = lens[b][h]
                if n == 0:
                    continue
                at = _row_tokens(c, s, b, h, torch.arange(n, device="cuda"))
                heads = slice(h * group, (h + 1) * group)
                logits = s["q"][b, heads].double() @ kf[at].double().T / math.sqrt(d)
                lse[b, heads] = torch.logsumexp(logits, 1)
                prob = torch.softmax(logits, 1)
                o[b, heads] = prob @ vf[at].double()
                if c["weights"]:
                    w[b, h, :n] = s["weights"][b, h, :n].double() + prob.sum(0)
        out = {"o": o, "lse": lse}
        if c["weights"]:
            out["weights"] = w
        return out
    k, v = kf.double(), vf.double()
    if c["op"] == "append":
        weights, positions, lens_out = s["weights"].double(), s["positions"].long(), s["lens"].long()
        lens, counts, start = s["lens"].tolist(), s["counts"].tolist(), s["start"].tolist()
        for b in range(c["batch"]):
            for h in range(c["hkv"]):
                n, m = lens[b][h], counts[b]
                at = _row_tokens(c, s, b, h, n + torch.arange(m, device="cuda"))
                k[at], v[at] = s["k"][b, h, :m].double(), s["v"][b, h, :m].double()
                weights[b, h, n:n + m] = 0
                positions[b, h, n:n + m] = start[b] + torch.arange(m, device="cuda")
                lens_out[b, h] = n + m
        return {"lens": lens_out, "k": k.view(s["k_pages"].shape), "v": v.view(s["v_pages"].shape), "weights": weights,
                "positions": positions}
    weights, positions, lens_out = s["weights_out"].double(), s["positions_out"].long(), s["lens"].long()
    lens, old_w, old_p = s["lens"].tolist(), s["weights"].cpu().numpy(), s["positions"].cpu().numpy()
    for b in range(c["batch"]):
        for h in range(c["hkv"]):
            n = lens[b][h]
            m = min(n, s["keep"][h])
            p, x = old_p[b, h, :n], old_w[b, h, :n]
            forced = (p < SINKS) | (p > (p.max() if n else 0) - RECENT)
            chosen = set(sorted(range(n), key=lambda i: (not forced[i], 0 if forced[i] else -x[i], i))[:m])
            slots = list(range(m))
            into = [i for i in range(m) if i not in chosen]
            for i, j in zip(into, sorted(i for i in chosen if i >= m)):
                slots[i] = j
            slots = torch.tensor(slots, device="cuda", dtype=torch.long)
            at = _row_tokens(c, s, b, h, slots)
            to = _row_tokens(c, s, b, h, torch.arange(m, device="cuda"))
            k[to], v[to] = kf[at].double(), vf[at].double()
            weights[b, h, :m] = s["weights"][b, h][slots].double()
            positions[b, h, :m] = s["positions"][b, h][slots].long()
            lens_out[b, h] = m
    return {"lens": lens_out, "k": k.view(s["k_pages"].shape), "v": v.view(s["v_pages"].shape), "weights": weights,
            "positions": positions}
