"""Cases of the operators that take prompts and new tokens into a paged cache, with their plain forms.

  pages    from the numbers of new tokens: which pages every (sequence, KV head) row gets or gives back, and the slot of
           every new token, so that rows grow, shrink and end without the host;
  rotary   rotates queries and keys by their positions (half or interleaved pairs, a part of the head, frequencies scaled
           for long contexts) and, with a cache, stores rotated keys and values in the new tokens' slots;
  packed   causal softmax attention of packed sequences of different lengths, grouped query heads; a sequence may have
           more keys than queries (a chunk of a prompt: its queries are the last ones).

What a run leaves alone (rows behind the last sequence, slots that receive no token) is part of its outputs.
"""
import math

import torch

own = False

PAGES = (16, 32, 64, 128, 256)
HEADS = ((8, 2, 64), (16, 16, 64), (32, 8, 128), (28, 4, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128))
# how frequencies are scaled for contexts longer than those trained on
SCALING = {
    "none": None,
    "linear": {"type": "linear", "factor": 4.0},
    "ntk": {"type": "ntk", "factor": 4.0},
    "wavelength": {"type": "wavelength", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192},
    "yarn": {"type": "yarn", "factor": 4.0, "original": 32768, "beta_fast": 32.0, "beta_slow": 1.0},
}


def _packed(name, batch, hq, hkv, d, lo, hi, past_lo=0, past_hi=0, pad=0):
    return {"name": name, "op": "packed", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "lo": lo, "hi": hi,
            "past_lo": past_lo, "past_hi": past_hi, "pad": pad}


def _rotary(name, tokens, hq, hkv, d, rot, interleaved, scaling, far, store, page=64, fused=True):
    return {"name": name, "op": "rotary", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "far": far, "store": store, "page": page, "fused": fused}


def _pages(name, batch, hkv, page, held_lo, held_hi, lo, hi, ended=0.0, spare=0, tight=False):
    return {"name": name, "op": "pages", "batch": batch, "hkv": hkv, "page": page, "held_lo": held_lo, "held_hi": held_hi,
            "lo": lo, "hi": hi, "ended": ended, "spare": spare, "tight": tight}


def listed():
    return [
        # one user's question: latency
        _packed("packed_chat", 1, 32, 8, 128, 41, 41),
        # the small model's heads, many prompts, none of them long
        _packed("packed_d64", 24, 8, 2, 64, 1, 1024),
        # a server's batch of prompts of any length, padded to the batch's capacity
        _packed("packed_batch", 16, 28, 4, 128, 1, 4096, pad=77),
        # chunks of two long prompts, their keys so far before them
        _packed("packed_chunk", 2, 64, 8, 128, 509, 509, 32768, 65536),
        # one whole long prompt
        _packed("packed_long", 1, 32, 8, 128, 32768, 32768),
        # a decode step's tokens, keys and values to their slots: latency
        _rotary("rotary_step", 64, 32, 8, 128, 128, False, "none", 8000, True, page=16),
        # a chunk of prompts, half of each head rotated in interleaved pairs, from a fused projection
        _rotary("rotary_part", 2049, 28, 4, 128, 64, True, "linear", 32768, False),
        # a whole prompt into the cache, frequencies scaled by wavelength
        _rotary("rotary_prompt", 32767, 32, 8, 128, 128, False, "wavelength", 0, True),
        # a chunk a million tokens into its context, the small model's heads
        _rotary("rotary_far", 4096, 8, 2, 64, 64, False, "yarn", 1 << 20, False, fused=False),
        # a decode step: one token a sequence, now and then a page
        _pages("pages_step", 64, 8, 16, 1, 8000, 1, 1),
        # prompts admitted to empty rows
        _pages("pages_prompts", 16, 8, 64, 0, 0, 1, 8192),
        # after evictions, some sequences ended: spare pages return and serve the next chunks
        _pages("pages_mixed", 32, 4, 32, 0, 16384, 0, 2048, ended=0.25, spare=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("packed", "packed", "rotary", "pages"))
    hq, hkv, d = rng.choice(HEADS)
    if op == "packed":
        batch = _log(rng, 1, 48)
        # no more work than the largest listed case: 4 * d * hq * sum of len^2 / 2
        most = 0.7 * math.sqrt(2 * 2.1e12 / (d * hq * batch))
        hi = _log(rng, 1, max(2, min(32768, most)))
        past = 0
        if rng.random() < 0.4:
            past = _log(rng, 1, max(2, min(65536, 1e12 / (d * hq * batch * hi), (1 << 28) / (batch * hkv * d))))
        c = _packed("", batch, hq, hkv, d, hi if rng.random() < 0.3 else rng.randint(0, hi), hi, rng.randint(0, past), past,
                    rng.choice((0, 0, rng.randint(1, 200))))
    elif op == "rotary":
        tokens = _log(rng, 1, min(32768, (1 << 28) // ((hq + hkv) * d)))
        rot = d if rng.random() < 0.5 else 16 * rng.randint(1, d // 16)
        c = _rotary("", tokens, hq, hkv, d, rot, rng.random() < 0.4, rng.choice(sorted(SCALING)), _log(rng, 1, 1 << 21),
                    rng.random() < 0.6, rng.choice(PAGES), rng.random() < 0.6)
    else:
        batch = _log(rng, 1, 256)
        page = rng.choice(PAGES)
        most = max(2, min(16384, (1 << 20) // (batch * hkv)))
        held = rng.choice((0, _log(rng, 1, most)))
        hi = 1 if rng.random() < 0.4 else _log(rng, 1, most)
        c = _pages("", batch, hkv, page, rng.randint(0, held), held, hi if rng.random() < 0.3 else rng.randint(0, hi), hi,
                   rng.choice((0.0, 0.2)), rng.choice((0, rng.randint(1, 24))), rng.random() < 0.2)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
BF16 = {"dtype": torch.bfloat16, "device": "cuda"}
BASE = 500000.0


def _lengths(b, lo, hi, g):
    """Lengths of a batch, the seed's own in their order, the case's in their sum."""
    return torch.randint(lo, hi + 1, (b,), generator=torch.Generator().manual_seed(b))[torch.randperm(b, generator=g)]


def _packed_inputs(c, s, g, opt):
    b, hq, h, d = c["batch"], c["hq"], c["hkv"], c["d"]
    n, past = _lengths(b, c["lo"], c["hi"], g), _lengths(b, c["past_lo"], c["past_hi"], g)
    s["n"], s["m"] = n.tolist(), (n + past).tolist()
    zero = torch.zeros(1, dtype=torch.int64)
    cu_q, cu_k = torch.cat((zero, n.cumsum(0))).int(), torch.cat((zero, (n + past).cumsum(0))).int()
    tq, tk = max(1, int(cu_q[-1]) + c["pad"]), max(1, int(cu_k[-1]) + c["pad"])
    s["cu_q"] = cu_q.cuda()
    s["cu_k"] = s["cu_q"] if c["past_hi"] == 0 else cu_k.cuda()
    # heads of differing sharpness, as the prefill inputs have
    sharp = torch.exp(torch.rand(hq, 1, **opt) * 1.4 - 0.7)
    s["q"] = (torch.randn(tq, hq, d, **opt) * sharp).bfloat16()
    s["k"] = torch.randn(tk, h, d, dtype=torch.bfloat16, **opt)
    s["v"] = torch.randn(tk, h, d, dtype=torch.bfloat16, **opt)
    s["o"] = torch.zeros(tq, hq, d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(tq, hq, device="cuda")


def _rotary_inputs(c, s, g, opt):
    t, hq, h, d = c["tokens"], c["hq"], c["hkv"], c["d"]
    if c["fused"]:
        qkv = torch.randn(t, hq + 2 * h, d, dtype=torch.bfloat16, **opt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
    else:
        s["q"], s["k"], s["v"] = (torch.randn(t, x, d, dtype=torch.bfloat16, **opt) for x in (hq, h, h))
    # a run of consecutive positions, or one far position a sequence where there are few tokens
    if t <= 256:
        s["positions"] = torch.randint(0, max(1, c["far"]), (t,), dtype=torch.int32, **opt)
    else:
        s["positions"] = (torch.arange(t, device="cuda") + max(0, c["far"] - t)).int()
    s["q_out"], s["k_out"] = torch.zeros(t, hq, d, **BF16), torch.zeros(t, h, d, **BF16)
    if c["store"]:
        page = c["page"]
        pages = -(-t // page)
        s["k_pages"] = torch.zeros(h * pages + 1, page, d, **BF16)
        s["v_pages"] = torch.zeros(h * pages + 1, page, d, **BF16)
        s["table"] = torch.randperm(h * pages + 1, **opt)[:h * pages].view(1, h, pages).int().contiguous()
        s["lens"] = torch.zeros(1, h, dtype=torch.int32, device="cuda")
        at = torch.arange(t, device="cuda")
        s["slots"] = s["table"][0].long()[:, at // page] * page + at % page
        # a few tokens have no slot (a row of the batch that is not active)
        s["slots"][:, torch.rand(t, **opt) < 0.02] = -1


def _pages_inputs(c, s, g, opt):
    b, h, page = c["batch"], c["hkv"], c["page"]
    held = torch.randint(c["held_lo"], c["held_hi"] + 1, (b, h if c["spare"] else 1), generator=g).expand(b, h)
    counts = _lengths(b, c["lo"], c["hi"], g)
    need = (held + page - 1) // page
    # rows that eviction cut hold fewer tokens than their pages could
    owned = need + (torch.randint(0, c["spare"] + 1, (b, h), generator=g) if c["spare"] else 0)
    max_pages = -(-(c["held_hi"] + max(c["hi"], page * c["spare"], 1)) // page)
    used, capacity = int(owned.sum()), b * h * max_pages + 100
    wanted = int(((held + counts[:, None] + page - 1) // page - owned).clamp(min=0).sum())
    free = wanted // 2 if c["tight"] else wanted + 100
    perm = torch.randperm(capacity, generator=g).int()
    table = torch.zeros(b, h, max_pages, dtype=torch.int32)
    mine = torch.arange(max_pages) < owned[..., None]
    table[mine] = perm[:used]
    s["table"] = table.cuda()
    s["lens"], s["owned"] = held.int().contiguous().cuda(), owned.int().contiguous().cuda()
    s["free"] = torch.zeros(capacity, dtype=torch.int32)
    s["free"][:free] = perm[used:used + free]
    s["free"] = s["free"].cuda()
    s["free_count"] = torch.tensor([free], dtype=torch.int32, device="cuda")
    s["cu"] = torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0))).int().cuda()
    s["total"] = max(1, int(counts.sum()))
    s["ended"] = (torch.rand(b, generator=g) < c["ended"]).cuda()
    s["start"] = (held.amax(1) + torch.randint(0, 1000, (b,), generator=g)).int().cuda()
    s["slots"] = torch.zeros(h, s["total"], dtype=torch.int64, device="cuda")
    s["positions"] = torch.zeros(s["total"], dtype=torch.int32, device="cuda")
    for name, like in (("lens_out", "lens"), ("owned_out", "owned"), ("free_out", "free_count"), ("start_out", "start"),
                       ("granted", "start")):
        s[name] = torch.zeros_like(s[like])


def _inputs(c, seed):
    g = torch.Generator().manual_seed(seed * 6151 + 29)
    opt = {"device": "cuda", "generator": torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)}
    s = {}
    {"packed": _packed_inputs, "rotary": _rotary_inputs, "pages": _pages_inputs}[c["op"]](c, s, g, opt)
    return s


def prepare(case, seed):
    s, c = _inputs(case, seed), case
    s["case"] = c
    if not own and c["op"] == "rotary":
        s["freq"], s["factor"] = _frequencies(c["rot"], SCALING[c["scaling"]])
    if own:
        import head_heterogeneous_block_gb300 as sa
        if c["op"] == "packed":
            s["layer"] = sa.PackedAttention(c["hq"], c["hkv"], c["d"], tokens=s["q"].shape[0], batch=c["batch"])
        elif c["op"] == "rotary":
            s["rotary"] = sa.Rotary(c["d"], rot_dim=c["rot"], base=BASE, interleaved=c["interleaved"],
                                    scaling=SCALING[c["scaling"]])
            if c["store"]:
                s["cache"] = sa.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["lens"])
        else:
            s["pool"] = sa.PagePool(s["table"], s["lens"], c["page"], free_pages=s["free"], free_count=s["free_count"],
                                    owned=s["owned"])
    return s


# ---------------------------------------------------------------- plain forms
def _frequencies(rot, scaling):
    """Radians a position of each pair, in 64 bits, and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    kind = scaling["type"] if scaling else "none"
    base = BASE
    if kind == "ntk" and rot > 2:
        base *= scaling["factor"] ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if kind == "linear":
        return f / scaling["factor"], 1.0
    if kind == "wavelength":
        # turns over the original context: up to `low` slowed down, from `high` on kept, a blend between
        turns = f * scaling["original"] / (2 * math.pi)
        keep = ((turns - scaling["low"]) / (scaling["high"] - scaling["low"])).clamp(0, 1)
        return f * keep + f / scaling["factor"] * (1 - keep), 1.0
    if kind == "yarn":
        def pair(beta):
            return rot * math.log(scaling["original"] / (beta * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair(scaling["beta_fast"])), 0)
        hi = min(math.ceil(pair(scaling["beta_slow"])), rot - 1)
        slow = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - slow) + f / scaling["factor"] * slow, 0.1 * math.log(scaling["factor"]) + 1.0
    return f, 1.0


def _plain_rotary(s):
    c = s["case"]
    rot = c["rot"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = (angle.cos() * s["factor"]).float()[:, None], (angle.sin() * s["factor"]).float()[:, None]
    for name in ("q", "k"):
        x = s[name].float()
        y = x.clone()
        if c["interleaved"]:
            x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        else:
            x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        s[name + "_out"].copy_(y)
    out = {"q": s["q_out"], "k": s["k_out"]}
    if c["store"]:
        there = (s["slots"] >= 0).flatten()
        at = s["slots"].flatten()[there]
        for name, x in (("k_pages", s["k_out"]), ("v_pages", s["v"])):
            s[name].view(-1, c["d"])[at] = x.transpose(0, 1).reshape(-1, c["d"])[there]
            out[name] = s[name]
    return out


def _plain_packed(s):
    c = s["case"]
    group, d = c["hq"] // c["hkv"], c["d"]
    scale = 1.0 / math.sqrt(d)
    q0 = k0 = 0
    for n, m in zip(s["n"], s["m"]):
        step = max(1, (1 << 27) // max(1, m * group))
        for a in range(0, n, step):
            e = min(n, a + step)
            seen = e + m - n                                       # keys that the chunk's last query sees
            live = torch.arange(seen, device="cuda") <= torch.arange(a, e, device="cuda")[:, None] + (m - n)
            for h in range(c["hkv"]):
                heads = slice(h * group, (h + 1) * group)
                k, v = s["k"][k0:k0 + seen, h].float(), s["v"][k0:k0 + seen, h].float()
                x = s["q"][q0 + a:q0 + e, heads].float().transpose(0, 1) @ k.T * scale
                x = torch.where(live, x, -math.inf)
                top = x.amax(-1, keepdim=True)
                x = torch.exp(x - top)
                total = x.sum(-1, keepdim=True)
                s["o"][q0 + a:q0 + e, heads] = ((x @ v) / total).transpose(0, 1).bfloat16()
                s["lse"][q0 + a:q0 + e, heads] = (top + total.log())[..., 0].T
        q0, k0 = q0 + n, k0 + m
    return {"o": s["o"], "lse": s["lse"]}


def _plain_pages(s):
    c = s["case"]
    b, h, page = c["batch"], c["hkv"], c["page"]
    cu, ended = s["cu"].long(), s["ended"]
    counts = cu[1:] - cu[:-1]
    held = torch.where(ended[:, None], 0, s["lens"].long())
    owned = s["owned"].long()
    need = (held + counts[:, None] + page - 1) // page
    back, wanted = (owned - need).clamp(min=0), (need - owned).clamp(min=0)
    old_free = s["free_count"].long()
    entry = torch.arange(s["table"].shape[-1], device="cuda")
    spare = (entry >= need[..., None]) & (entry < owned[..., None])
    # the free pages and, above them, those that come back
    back_at = torch.where(spare.flatten(), old_free + spare.flatten().long().cumsum(0) - 1, 0)
    stack = torch.zeros(s["free"].numel() + 1, dtype=torch.int64, device="cuda")
    stack[:-1] = torch.where(torch.arange(s["free"].numel(), device="cuda") < old_free, s["free"].long(), 0)
    stack.scatter_add_(0, back_at, torch.where(spare.flatten(), s["table"].flatten().long(), 0))
    total = old_free + back.sum()
    per_seq = wanted.sum(1)
    ok = (per_seq == 0) | (per_seq.cumsum(0) <= total)
    taken = torch.where(ok[:, None], wanted, 0)
    first = (taken.flatten().cumsum(0) - taken.flatten()).view(b, h)
    fresh = (entry >= owned[..., None]) & (entry < (owned + taken)[..., None])
    nth = first[..., None] + entry - owned[..., None]
    handed = stack[(total - 1 - nth).clamp(0, stack.numel() - 1)]
    table = torch.where(fresh, handed, s["table"].long())
    s["table"].copy_(table)
    left = total - taken.sum()
    where = torch.arange(s["free"].numel(), device="cuda")
    s["free"].copy_(torch.where((where >= old_free) & (where < left), stack[:-1], s["free"].long()))
    s["free_out"].copy_(left)
    s["owned_out"].copy_(owned - back + taken)
    granted = torch.where(ok, counts, 0)
    s["granted"].copy_(granted)
    s["lens_out"].copy_(held + granted[:, None])
    begin = torch.where(ended, 0, s["start"].long())
    s["start_out"].copy_(begin + granted)
    # every new token's sequence and number in it
    t = torch.arange(s["total"], device="cuda")
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=b - 1)
    i = t - cu[seq]
    new = i < granted[seq]
    slot = held[seq].T + i                                          # [h, tokens]
    number = table[seq].permute(1, 0, 2).gather(-1, (slot // page).clamp(max=table.shape[-1] - 1)[..., None])[..., 0]
    s["slots"].copy_(torch.where(new, number * page + slot % page, -1))
    s["positions"].copy_(torch.where(new, begin[seq] + i, 0))
    return _page_outputs(s)


def _page_outputs(s):
    return {"table": s["table"], "lens": s["lens_out"], "owned": s["owned_out"], "free": s["free"], "free_count": s["free_out"],
            "start": s["start_out"], "granted": s["granted"], "slots": s["slots"], "positions": s["positions"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"packed": _plain_packed, "rotary": _plain_rotary, "pages": _plain_pages}[c["op"]](s)
    if c["op"] == "packed":
        s["layer"](s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["o"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "rotary":
        out = {"q": s["q_out"], "k": s["k_out"]}
        if c["store"]:
            s["rotary"].store(s["q"], s["k"], s["v"], s["positions"], s["cache"], s["slots"], q_out=s["q_out"],
                              k_out=s["k_out"])
            out["k_pages"], out["v_pages"] = s["k_pages"], s["v_pages"]
        else:
            s["rotary"](s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"])
        return out
    s["pool"].grow(s["slots"], cu=s["cu"], ended=s["ended"], start=s["start"], positions=s["positions"], granted=s["granted"],
                   lens_out=s["lens_out"], owned_out=s["owned_out"], free_count_out=s["free_out"], start_out=s["start_out"])
    return _page_outputs(s)


def work(case):
    c = case
    h = c["hkv"]
    if c["op"] == "rotary":
        t, d = c["tokens"], c["d"]
        moved = t * (c["hq"] + h) * d * 4 + t * 4
        if c["store"]:
            moved += t * h * (3 * d * 2 + 8)
        return {"bytes": moved, "flops": t * (c["hq"] + h) * c["rot"] * 3}
    if c["op"] == "packed":
        n, past = (c["lo"] + c["hi"]) / 2, (c["past_lo"] + c["past_hi"]) / 2
        # mean of n^2 over the drawn lengths
        square = n * n + ((c["hi"] - c["lo"] + 1) ** 2 - 1) / 12
        seen = c["batch"] * (square / 2 + n / 2 + n * past)
        return {"bytes": c["batch"] * (n * c["hq"] * (4 * c["d"] + 4) + (n + past) * h * 4 * c["d"]),
                "flops": seen * c["hq"] * 4 * c["d"]}
    rows = c["batch"] * h
    new = (c["lo"] + c["hi"]) / 2
    pages = rows * max(1 if new else 0, new / c["page"])            # entries read or written
    back = rows * c["spare"] / 2 + c["ended"] * rows * (c["held_lo"] + c["held_hi"]) / 2 / c["page"]
    return {"bytes": rows * 16 + c["batch"] * 20 + (pages + back) * 8 + rows * new * 8 + c["batch"] * new * 4, "flops": 0}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    c, s = case, _inputs(case, seed)
    return {"packed": _exact_packed, "rotary": _exact_rotary, "pages": _exact_pages}[c["op"]](c, s)


def _exact_packed(c, s):
    d, group = c["d"], c["hq"] // c["hkv"]
    o, lse = s["o"].double(), s["lse"].double()
    at_q = at_k = 0
    for n, m in zip(s["n"], s["m"]):
        for kv in range(c["hkv"]):
            keys, values = s["k"][at_k:at_k + m, kv].double(), s["v"][at_k:at_k + m, kv].double()
            for a in range(0, n, 1024):
                z = min(n, a + 1024)
                far = z + m - n
                for head in range(kv * group, (kv + 1) * group):
                    logits = s["q"][at_q + a:at_q + z, head].double() @ keys[:far].T / math.sqrt(d)
                    later = torch.ones(z - a, far, dtype=torch.bool, device="cuda").triu(a + m - n + 1)
                    logits.masked_fill_(later, -math.inf)
                    lse[at_q + a:at_q + z, head] = torch.logsumexp(logits, 1)
                    o[at_q + a:at_q + z, head] = torch.softmax(logits, 1) @ values[:far]
        at_q, at_k = at_q + n, at_k + m
    return {"o": o, "lse": lse}


def _exact_rotary(c, s):
    rot = c["rot"]
    scaling = SCALING[c["scaling"]] or {"type": "none"}
    freq, factor = [], 1.0
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(BASE))
        if scaling["type"] == "linear":
            f /= scaling["factor"]
        elif scaling["type"] == "ntk" and rot > 2:
            f = math.exp(-2.0 * i / rot * (math.log(BASE) + rot / (rot - 2) * math.log(scaling["factor"])))
        elif scaling["type"] == "wavelength":
            wave = 2 * math.pi / f
            if wave > scaling["original"] / scaling["low"]:
                f /= scaling["factor"]
            elif wave > scaling["original"] / scaling["high"]:
                part = (scaling["original"] / wave - scaling["low"]) / (scaling["high"] - scaling["low"])
                f = (1 - part) * f / scaling["factor"] + part * f
        elif scaling["type"] == "yarn":
            edge = [rot / 2 * math.log(scaling["original"] / (x * 2 * math.pi)) / math.log(BASE)
                    for x in (scaling["beta_fast"], scaling["beta_slow"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / scaling["factor"] * ramp + f * (1 - ramp)
            factor = 1.0 + 0.1 * math.log(scaling["factor"])
        freq.append(f)
    turn = torch.exp(1j * s["positions"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")) * factor
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous()) * turn[:, None]
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn[:, None]
            y[..., :rot] = torch.cat((z.real, z.imag), -1)
        out[name] = y
    if c["store"]:
        for name, x in (("k_pages", out["k"]), ("v_pages", s["v"].double())):
            pool = s[name].double()
            for kv in range(c["hkv"]):
                has = s["slots"][kv] >= 0
                at = s["slots"][kv][has]
                pool[at // c["page"], at % c["page"]] = x[:, kv][has]
            out[name] = pool
    return out


def _exact_pages(c, s):
    page, h = c["page"], c["hkv"]
    a = {k: s[k].cpu().numpy().copy() for k in ("table", "lens", "owned", "free", "cu", "ended", "start", "granted", "slots",
                                                "positions")}
    count = int(s["free_count"][0])
    stack = a["free"][:count].tolist()
    counts = [int(a["cu"][b + 1] - a["cu"][b]) for b in range(c["batch"])]
    held = [[0 if a["ended"][b] else int(a["lens"][b, g]) for g in range(h)] for b in range(c["batch"])]
    start = [0 if a["ended"][b] else int(a["start"][b]) for b in range(c["batch"])]
    need = [[-(-(held[b][g] + counts[b]) // page) for g in range(h)] for b in range(c["batch"])]
    for b in range(c["batch"]):                                     # spare pages first
        for g in range(h):
            while a["owned"][b, g] > need[b][g]:
                a["owned"][b, g] -= 1
            had = int(s["owned"][b, g])
            stack += a["table"][b, g, a["owned"][b, g]:had].tolist()
    promised = 0
    room = len(stack)
    for b in range(c["batch"]):
        more = sum(max(0, need[b][g] - int(a["owned"][b, g])) for g in range(h))
        promised += more
        given = counts[b] if more == 0 or promised <= room else 0
        at = int(a["cu"][b])
        for g in range(h):
            while given and a["owned"][b, g] < need[b][g]:
                a["table"][b, g, a["owned"][b, g]] = stack.pop()
                a["owned"][b, g] += 1
            for i in range(counts[b]):
                slot = held[b][g] + i
                a["slots"][g, at + i] = int(a["table"][b, g, slot // page]) * page + slot % page if i < given else -1
            a["lens"][b, g] = held[b][g] + given
        a["granted"][b], a["start"][b] = given, start[b] + given
        for i in range(counts[b]):
            a["positions"][at + i] = start[b] + i if i < given else 0
    if a["cu"][-1] == 0:                                            # the map's one entry belongs to no sequence
        a["slots"][:], a["positions"][:] = -1, 0
    if len(stack) > count:
        a["free"][count:len(stack)] = stack[count:]
    out = {k: torch.from_numpy(a[k]).cuda() for k in ("table", "lens", "owned", "free", "start", "granted", "slots", "positions")}
    out["free_count"] = torch.tensor([len(stack)], dtype=torch.int32, device="cuda")
    return out
