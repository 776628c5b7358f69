"""The serving-path operators around the row select, as cases that can be timed
and compared: each case is run either by this package's kernels (``own``) or in
the operator's plain form, elementary torch operations in 32 bits.

The path is one step of sparse attention over a paged cache: place a batch's
new tokens in the cache (assign_slots), score every cached key for every query
token (indexer_logits, indexer_logits_paged), select rows from the scores
(topk_rows, emit_rows: measured elsewhere), attend over the selected rows or
over the whole paged prefix with the keys and values of one shared latent
vector a token (latent_attend_rows, latent_attend_paged), and join the partial
results of ranks that each own a part of the rows (merge_attend_rank_major).
"""

import math

import torch

own = False

ROPE = 64   # positional part of a latent cache row; the latent part precedes it
DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # A pure decode step: 64 requests, one new token each. Latency counts.
        {"name": "slots_decode", "op": "slots", "reqs": 64, "new": 1, "ctx": 8192, "block": 64, "pad": 0},
        # A mixed step: decodes and prompt chunks in one padded batch, small pages.
        {"name": "slots_mixed", "op": "slots", "reqs": 509, "new": 257, "ctx": 16384, "block": 16, "pad": 1000},
        # Prompt chunk of odd length, bf16 index keys.
        {"name": "logits_bf16", "op": "logits", "rows": 333, "cols": 8191, "heads": 32, "dim": 128,
         "e4m3": False},
        # Prompt chunk against a long prefix, 8-bit index keys: the most work.
        {"name": "logits_e4m3", "op": "logits", "rows": 1024, "cols": 16384, "heads": 64, "dim": 128,
         "e4m3": True},
        # A decode step over long paged contexts, 8-bit keys.
        {"name": "logits_paged_decode", "op": "logits_paged", "reqs": 64, "each": 1, "ctx": 32768,
         "heads": 64, "dim": 128, "block": 64, "e4m3": True},
        # Few requests with three tokens each (two of them drafted), bf16 keys, small pages.
        {"name": "logits_paged_draft", "op": "logits_paged", "reqs": 7, "each": 3, "ctx": 9001,
         "heads": 32, "dim": 128, "block": 16, "e4m3": False},
        # Decode over the rows that the select kept; heads of one of several ranks.
        {"name": "rows_decode", "op": "rows", "rows": 64, "heads": 16, "k": 2048, "ctx": 8192,
         "reqs": 64, "latent": 512, "block": 64},
        # A prompt chunk: every token has its own selected rows of one context, all heads.
        {"name": "rows_prefill", "op": "rows", "rows": 1024, "heads": 128, "k": 2048, "ctx": 16384,
         "reqs": 1, "latent": 512, "block": 64},
        # Dense decode over ragged paged contexts, all heads.
        {"name": "paged_decode", "op": "paged", "reqs": 32, "each": 1, "ctx": 16384, "heads": 128,
         "latent": 512, "block": 64, "tree": False},
        # Trees of drafted tokens over a cache, a few requests, few heads. Latency counts.
        {"name": "paged_tree", "op": "paged", "reqs": 6, "each": 8, "ctx": 4001, "heads": 16,
         "latent": 512, "block": 16, "tree": True},
        # A decode step's partial results of 4 ranks.
        {"name": "merge_decode", "op": "merge", "world": 4, "rows": 64, "heads": 16, "dim": 512},
        # A prompt chunk's partial results of 8 ranks, all heads.
        {"name": "merge_prefill", "op": "merge", "world": 8, "rows": 1000, "heads": 128, "dim": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "logits", "logits_paged", "rows", "paged", "merge"])
    heads = rng.choice([1, 8, 16, 20, 32, 40, 64, 96, 128])
    latent = rng.choice([256, 512, 512, 512])
    block = rng.choice([1, 16, 32, 48, 64, 128])
    if op == "slots":
        return {"op": op, "reqs": _log(rng, 1, 1000), "new": _log(rng, 1, 300), "ctx": _log(rng, 1, 20000),
                "block": max(block, 16), "pad": rng.choice([0, 1, 77, 2048])}
    if op == "logits":
        rows, cols = _log(rng, 1, 1024), _log(rng, 17, 16384)
        return {"op": op, "rows": rows, "cols": cols, "heads": rng.choice([1, 8, 24, 32, 64]),
                "dim": rng.choice([64, 128, 128]), "e4m3": rng.random() < 0.5}
    if op == "logits_paged":
        reqs, each = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 5])
        ctx = _log(rng, 1, max(2, min(32768, 64 * 32768 // (reqs * each))))
        return {"op": op, "reqs": reqs, "each": each, "ctx": ctx, "heads": rng.choice([1, 8, 24, 32, 64]),
                "dim": rng.choice([64, 128, 128]), "block": block, "e4m3": rng.random() < 0.5}
    if op == "rows":
        rows, k = _log(rng, 1, 1000), rng.choice([1, 100, 512, 1000, 2048])
        reqs = rng.choice([1, rows])
        ctx = _log(rng, 16, 16384 if reqs == 1 else max(32, min(16384, 1 << 20 // reqs)))
        return {"op": op, "rows": rows, "heads": heads, "k": k, "ctx": ctx, "reqs": reqs,
                "latent": latent, "block": block}
    if op == "paged":
        reqs, tree = _log(rng, 1, 32), rng.random() < 0.4
        each = rng.choice([2, 5, 8, 17, 64]) if tree else rng.choice([1, 1, 1, 2, 4, 100])
        ctx = _log(rng, 1, max(2, min(16384, 500000 // (reqs * each))))
        return {"op": op, "reqs": reqs, "each": each, "ctx": ctx, "heads": heads, "latent": latent,
                "block": block, "tree": tree}
    return {"op": op, "world": rng.choice([1, 2, 3, 4, 8]), "rows": _log(rng, 1, 1000), "heads": heads,
            "dim": latent}


# --------------------------------------------------------------------------- inputs

def _ints(g, lo, hi, n):
    """n whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int64)


def _table(g, reqs, cols):
    """Block tables of requests whose pages lie anywhere in the cache."""
    return torch.randperm(reqs * cols, generator=g, device=DEV).to(torch.int32).view(reqs, cols)


def _spread(g, lo, hi, n):
    """n lengths spread over [lo, hi] in random order: ragged, with the same sum for every seed."""
    at = torch.arange(n, device=DEV) % (hi - lo + 1)
    return (hi - at)[torch.randperm(n, generator=g, device=DEV)]


def _contexts(g, case):
    """Cached lengths: ragged, one of them the longest."""
    ctx = _ints(g, case["ctx"] // 2, case["ctx"], case["reqs"])
    ctx[0] = case["ctx"]
    return ctx


def _as(x, e4m3):
    return x.to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)


def _prepare_slots(c, g):
    new = _spread(g, 1, c["new"], c["reqs"])
    ctx = _ints(g, 0, c["ctx"], c["reqs"])
    cols = -(-(c["ctx"] + c["new"]) // c["block"])
    have = -(-ctx // c["block"])
    spare = c["reqs"] * (c["new"] // c["block"] + 2)
    blocks = torch.randperm(c["reqs"] * cols + spare, generator=g, device=DEV).to(torch.int32)
    table, free = blocks[spare:].view(c["reqs"], cols).clone(), blocks[:spare].clone()
    table[torch.arange(cols, device=DEV)[None] >= have[:, None]] = -1
    tokens = int(new.sum()) + c["pad"]
    return {"ctx": ctx.int(), "new": new.int(), "tokens": tokens, "table": table, "free": free}


def _prepare_logits(c, g):
    q = _as(torch.randn(c["rows"], c["heads"], c["dim"], generator=g, device=DEV), c["e4m3"])
    keys = _as(torch.randn(c["cols"], c["dim"], generator=g, device=DEV), c["e4m3"])
    w = torch.randn(c["rows"], c["heads"], generator=g, device=DEV) * (c["heads"] * c["dim"]) ** -0.5
    scales = torch.rand(c["cols"], generator=g, device=DEV) + 0.5 if c["e4m3"] else None
    ends = torch.arange(c["rows"], device=DEV) + c["cols"] - c["rows"] + 1  # causal
    out = torch.zeros(c["rows"], c["cols"], device=DEV)
    return {"q": q, "keys": keys, "w": w, "scales": scales, "ends": ends.clamp(min=0).int(), "out": out}


def _prepare_logits_paged(c, g):
    reqs, each = c["reqs"], c["each"]
    ctx = _contexts(g, c)
    cols = -(-(c["ctx"] + each) // c["block"])
    cache_rows = reqs * cols * c["block"]
    rows = reqs * each
    q = _as(torch.randn(rows, c["heads"], c["dim"], generator=g, device=DEV), c["e4m3"])
    keys = _as(torch.randn(cache_rows, c["dim"], generator=g, device=DEV), c["e4m3"])
    w = torch.randn(rows, c["heads"], generator=g, device=DEV) * (c["heads"] * c["dim"]) ** -0.5
    scales = torch.rand(cache_rows, generator=g, device=DEV) + 0.5 if c["e4m3"] else None
    at = torch.arange(rows, device=DEV)
    req = at // each
    return {"q": q, "keys": keys, "w": w, "scales": scales, "req": req.int(), "cols": c["ctx"] + each,
            "ends": (ctx[req] + at % each + 1).int(), "table": _table(g, reqs, cols),
            "out": torch.zeros(rows, c["ctx"] + each, device=DEV)}


def _prepare_rows(c, g):
    rows, reqs, k = c["rows"], c["reqs"], c["k"]
    cols = -(-c["ctx"] // c["block"])
    table = _table(g, reqs, cols).long()
    cache = torch.randn(reqs * cols * c["block"], c["latent"] + ROPE, generator=g, device=DEV).bfloat16()
    q = torch.randn(rows, c["heads"], c["latent"] + ROPE, generator=g, device=DEV).bfloat16()
    at = torch.arange(rows, device=DEV)
    # One request: its last rows, causal. Many: one token each, ragged lengths.
    ends = (at + c["ctx"] - rows + 1).clamp(min=0) if reqs == 1 else _ints(g, 0, c["ctx"], rows)
    ends[-1] = c["ctx"]
    n = min(k, c["ctx"])
    ids = torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
    for r in range(0, rows, 256):
        key = torch.rand(min(256, rows - r), c["ctx"], generator=g, device=DEV)
        e = ends[r:r + 256, None]
        key.masked_fill_(torch.arange(c["ctx"], device=DEV)[None] >= e, -1.0)
        v, pos = key.topk(n, dim=1)
        req = (at[r:r + 256, None] if reqs > 1 else 0 * e)
        phys = table[req, pos // c["block"]] * c["block"] + pos % c["block"]
        ids[r:r + 256, :n] = torch.where(v >= 0, phys, -1).int()
    counts = ends.clamp(max=n).int()
    return {"q": q, "cache": cache, "ids": ids, "counts": counts, "scale": (128 + ROPE) ** -0.5}


def _prepare_paged(c, g):
    reqs, each = c["reqs"], c["each"]
    ctx = _contexts(g, c)
    new = _spread(g, max(1, each // 2), each, reqs)
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    tokens = int(starts[-1])
    cols = -(-(c["ctx"] + each) // c["block"])
    cache = torch.randn(reqs * cols * c["block"], c["latent"] + ROPE, generator=g, device=DEV).bfloat16()
    q = torch.randn(tokens, c["heads"], c["latent"] + ROPE, generator=g, device=DEV).bfloat16()
    tree = None
    if c["tree"]:  # each drafted token's parent is one before it; bit j: draft j is an ancestor or itself
        req = torch.repeat_interleave(torch.arange(reqs, device=DEV), new)
        own_at = (torch.arange(tokens, device=DEV) - starts[req]).tolist()
        pick = torch.rand(tokens, generator=g, device=DEV).tolist()
        first, masks = starts[req].tolist(), []
        for t in range(tokens):
            j = own_at[t]
            parent = masks[first[t] + int(pick[t] * j)] if j else 0
            masks.append(parent | (1 << j))
        tree = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
    return {"q": q, "cache": cache, "starts": starts.int(), "ctx": ctx.int(), "tree": tree,
            "table": _table(g, reqs, cols), "max_len": c["ctx"] + each, "scale": (128 + ROPE) ** -0.5}


def _prepare_merge(c, g):
    parts = torch.randn(c["world"], c["rows"], c["heads"], c["dim"], generator=g, device=DEV).bfloat16()
    lse = torch.randn(c["world"], c["rows"], c["heads"], generator=g, device=DEV) * 2 + 7
    lse[torch.rand(lse.shape, generator=g, device=DEV) < 0.02] = -math.inf  # ranks that own no row
    return {"parts": parts, "lse": lse}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    make = {"slots": _prepare_slots, "logits": _prepare_logits, "logits_paged": _prepare_logits_paged,
            "rows": _prepare_rows, "paged": _prepare_paged, "merge": _prepare_merge}[case["op"]]
    return {"case": case, **make(case, g)}


# --------------------------------------------------------------------------- plain forms

def _plain_slots(s):
    b, ctx, new, table = s["case"]["block"], s["ctx"].long(), s["new"].long(), s["table"]
    tokens, reqs = s["tokens"], ctx.numel()
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    have, need = (ctx + b - 1) // b, (ctx + new + b - 1) // b
    take = need - have
    first = take.cumsum(0) - take
    col = torch.arange(table.shape[1], device=DEV)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    src = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][src], table))
    at = torch.arange(tokens, device=DEV)
    req = torch.searchsorted(starts[1:], at, right=True)
    live = req < reqs
    r = req.clamp(max=reqs - 1)
    pos = ctx[r] + at - starts[r]
    slot = table[r, (pos // b).clamp(max=table.shape[1] - 1)].long() * b + pos % b
    return {"query_starts": starts.int(), "req_id": torch.where(live, req, -1).int(),
            "row_ends": torch.where(live, pos + 1, 0).int(), "slots": torch.where(live, slot, -1).int(),
            "used": take.sum().int().view(1), "block_table": table}


def _plain_logits(s):
    q, keys = s["q"].float(), s["keys"].float()
    rows, heads, dim = q.shape
    dots = (q.view(rows * heads, dim) @ keys.t().contiguous()).view(rows, heads, -1)
    x = torch.bmm(s["w"][:, None], dots.clamp_(min=0)).squeeze(1)
    if s["scales"] is not None:
        x = x * s["scales"]
    inside = torch.arange(keys.shape[0], device=DEV)[None] < s["ends"][:, None]
    s["out"].copy_(torch.where(inside, x, s["out"]))
    return s["out"]


def _plain_logits_paged(s):
    b, cols = s["case"]["block"], s["cols"]
    pos = torch.arange(cols, device=DEV)
    phys = s["table"][:, pos // b].long() * b + pos % b                    # [reqs, cols]
    q, keys = s["q"].float(), s["keys"][phys].float()                      # [reqs, cols, dim]
    rows, heads, dim = q.shape
    reqs = phys.shape[0]
    dots = torch.bmm(q.view(reqs, -1, dim), keys.transpose(1, 2).contiguous()).view(rows, heads, cols)
    x = torch.bmm(s["w"][:, None], dots.clamp_(min=0)).squeeze(1)
    if s["scales"] is not None:
        x = x * s["scales"][phys][s["req"].long()]
    inside = pos[None] < s["ends"][:, None]
    s["out"].copy_(torch.where(inside, x, s["out"]))
    return s["out"]


def _plain_attend(q, kv, keep, scale, latent):
    """q [n, heads, d], kv [n, keys, d] and keep [n, keys]: softmax(q kv' scale) over the kept keys,
    times their latent parts; rows that keep nothing give zeros and -inf."""
    x = torch.bmm(q.float(), kv.transpose(1, 2).contiguous()) * scale
    x = x.masked_fill_(~keep[:, None], -math.inf)
    m = x.amax(2, keepdim=True).clamp_(min=-3e38)
    p = (x - m).exp_()
    total = p.sum(2, keepdim=True)
    v = kv[:, :, :latent] * keep[:, :, None]
    out = torch.bmm(p, v) / total.clamp(min=1e-38)
    lse = torch.where(total > 0, m + total.log(), -math.inf).squeeze(2)
    return out.bfloat16(), lse


def _plain_rows(s):
    ids = s["ids"].long()
    keep = (ids >= 0) & (torch.arange(ids.shape[1], device=DEV)[None] < s["counts"][:, None])
    kv = s["cache"][ids.clamp(min=0)].float()
    return _plain_attend(s["q"], kv, keep, s["scale"], s["case"]["latent"])


def _plain_paged(s):
    b, n = s["case"]["block"], s["max_len"]
    starts, ctx = s["starts"].long(), s["ctx"].long()
    at = torch.arange(s["q"].shape[0], device=DEV)
    req = torch.searchsorted(starts[1:], at, right=True)
    idx = at - starts[req]
    pos = torch.arange(n, device=DEV)
    phys = s["table"][:, pos // b].long() * b + pos % b
    kv = s["cache"][phys].float()[req]
    draft = pos[None] - ctx[req][:, None]                                   # [tokens, n]
    if s["tree"] is None:
        keep = draft <= idx[:, None]
    else:
        bit = (s["tree"][:, None] >> draft.clamp(0, 63)) & 1
        new = starts[req + 1] - starts[req]
        keep = (draft < 0) | ((draft < new[:, None]) & (draft < 64) & (bit == 1))
    return _plain_attend(s["q"], kv, keep, s["scale"], s["case"]["latent"])


def _plain_merge(s):
    lse = s["lse"]
    m = lse.amax(0, keepdim=True).clamp(min=-3e38)
    w = (lse - m).exp()
    total = w.sum(0)
    out = (s["parts"].float() * w[..., None]).sum(0) / total.clamp(min=1e-38)[..., None]
    return out.bfloat16(), torch.where(total > 0, m[0] + total.log(), -math.inf)


# --------------------------------------------------------------------------- one pass

def run(state):
    c, s = state["case"], state
    if own:
        import row_top_select_amd as rts
        if c["op"] == "slots":
            m = rts.assign_slots(s["ctx"], s["new"], s["tokens"], s["table"], s["free"], c["block"])
            return {**m._asdict(), "block_table": s["table"]}
        if c["op"] == "logits":
            return rts.indexer_logits(s["q"], s["keys"], s["w"], key_scales=s["scales"], row_ends=s["ends"],
                                      out=s["out"])
        if c["op"] == "logits_paged":
            return rts.indexer_logits_paged(s["q"], s["keys"], s["w"], s["req"], s["ends"], s["table"],
                                            c["block"], s["cols"], key_scales=s["scales"], out=s["out"])
        if c["op"] == "rows":
            return rts.latent_attend_rows(s["q"], s["cache"], s["ids"], s["scale"], d_latent=c["latent"],
                                          counts=s["counts"])
        if c["op"] == "paged":
            return rts.latent_attend_paged(s["q"], s["cache"], s["starts"], s["ctx"], s["table"], c["block"],
                                           s["scale"], d_latent=c["latent"], tree=s["tree"],
                                           max_len=s["max_len"])
        return rts.merge_attend_rank_major(s["parts"], s["lse"])
    plain = {"slots": _plain_slots, "logits": _plain_logits, "logits_paged": _plain_logits_paged,
             "rows": _plain_rows, "paged": _plain_paged, "merge": _plain_merge}[c["op"]]
    return plain(s)


# --------------------------------------------------------------------------- floors

def work(case):
    """Each input once, each output once, and the products of the definition."""
    c = case
    if c["op"] == "slots":
        tokens = c["reqs"] * (c["new"] + 1) // 2 + c["pad"]
        fresh = c["reqs"] * (1 + c["new"] // (2 * c["block"]))
        return {"bytes": c["reqs"] * 12 + tokens * 16 + fresh * 8, "flops": 0}
    if c["op"] == "logits":
        size = 1 if c["e4m3"] else 2
        pairs = sum(max(0, c["cols"] - c["rows"] + 1 + i) for i in range(c["rows"]))
        return {"bytes": c["rows"] * c["heads"] * (c["dim"] * size + 4) + c["cols"] * c["dim"] * size + pairs * 4,
                "flops": pairs * c["heads"] * (2 * c["dim"] + 2)}
    if c["op"] == "logits_paged":
        size = 1 if c["e4m3"] else 2
        keys = c["reqs"] * c["ctx"] * 3 // 4
        rows = c["reqs"] * c["each"]
        pairs = keys * c["each"]
        return {"bytes": rows * c["heads"] * (c["dim"] * size + 4) + keys * (c["dim"] * size + 4) + pairs * 4,
                "flops": pairs * c["heads"] * (2 * c["dim"] + 2)}
    d = c.get("latent", 0) + ROPE
    if c["op"] == "rows":
        if c["reqs"] == 1:
            pairs = sum(min(c["k"], max(0, c["ctx"] - c["rows"] + 1 + i)) for i in range(c["rows"]))
            touched = min(c["ctx"], pairs)
        else:  # lengths are spread evenly over [0, ctx]
            k = min(c["k"], c["ctx"])
            pairs = touched = int(c["rows"] * k * (1 - k / (2 * c["ctx"])))
        return {"bytes": c["rows"] * c["heads"] * (d + c["latent"] + 2) * 2 + touched * d * 2 + pairs * 4,
                "flops": pairs * c["heads"] * 2 * (d + c["latent"])}
    if c["op"] == "paged":
        new = (max(1, c["each"] // 2) + c["each"]) / 2
        keys = c["reqs"] * c["ctx"] * 0.75
        rows = c["reqs"] * new
        return {"bytes": rows * c["heads"] * (d + c["latent"] + 2) * 2 + keys * d * 2,
                "flops": keys * new * c["heads"] * 2 * (d + c["latent"])}
    n = c["rows"] * c["heads"]
    return {"bytes": (c["world"] + 1) * n * (c["dim"] * 2 + 4), "flops": c["world"] * n * 2 * c["dim"]}


# --------------------------------------------------------------------------- 64 bits

def _exact_attention(q, kv, scale, latent):
    """One token's heads over the keys that it keeps."""
    if kv.shape[0] == 0:
        return q.new_zeros(q.shape[0], latent), q.new_full((q.shape[0],), -math.inf)
    z = (q @ kv.t()) * scale
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse[:, None]) @ kv[:, :latent], lse


def exact(case, seed):
    c = case
    if c["op"] == "slots":
        return None  # whole numbers: the plain form's are the definition's
    s = prepare(case, seed)
    if c["op"] in ("logits", "logits_paged"):
        out = s["out"].double()
        for t in range(out.shape[0]):
            e = int(s["ends"][t])
            if c["op"] == "logits":
                at = slice(0, e)
            else:
                p = torch.arange(e, device=DEV)
                page = s["table"][int(s["req"][t])].long()
                at = page[torch.div(p, c["block"], rounding_mode="floor")] * c["block"] + p.remainder(c["block"])
            per_head = torch.relu(s["keys"][at].double() @ s["q"][t].double().t())  # [keys, heads]
            score = per_head @ s["w"][t].double()
            out[t, :e] = score * s["scales"][at].double() if c["e4m3"] else score
        return out
    if c["op"] == "merge":
        lse = s["lse"].double()
        total = torch.logsumexp(lse, 0)
        share = torch.where(lse == -math.inf, torch.zeros_like(lse), torch.exp(lse - total))
        out = torch.zeros_like(s["parts"][0], dtype=torch.float64)
        for r in range(c["world"]):
            out += share[r][..., None] * s["parts"][r].double()
        return out, total
    outs, sums = [], []
    if c["op"] == "rows":
        for t in range(s["q"].shape[0]):
            ids = s["ids"][t, : int(s["counts"][t])].long()
            o, l = _exact_attention(s["q"][t].double(), s["cache"][ids[ids >= 0]].double(), s["scale"], c["latent"])
            outs.append(o)
            sums.append(l)
    else:
        starts, ctx = s["starts"].tolist(), s["ctx"].tolist()
        for r in range(c["reqs"]):
            n = ctx[r] + starts[r + 1] - starts[r]
            pos = torch.arange(n, device=DEV)
            page = s["table"][r].long()
            kv = s["cache"][page[torch.div(pos, c["block"], rounding_mode="floor")] * c["block"]
                            + pos.remainder(c["block"])].double()
            for t in range(starts[r], starts[r + 1]):
                seen = list(range(ctx[r]))
                mask = (2 << (t - starts[r])) - 1 if s["tree"] is None else int(s["tree"][t])
                seen += [ctx[r] + j for j in range(n - ctx[r]) if (mask >> j) & 1]
                o, l = _exact_attention(s["q"][t].double(), kv[seen], s["scale"], c["latent"])
                outs.append(o)
                sums.append(l)
    return torch.stack(outs), torch.stack(sums)
