"""The operators of a beam-search step over a paged cache, as cases that can be
timed and compared: each case is run either by this package's kernels (``own``)
or in the operator's plain form, elementary torch operations.

A step continues each request's hypotheses: score every token for every beam
and keep the best of them (beam_select), let the rows of the block table follow
the beams that were kept, with fresh blocks where two beams would write into the
same one (fork_blocks), copy those blocks (copy_blocks), and attend from the new
tokens over their cached keys and values (kv_attend_paged).  From time to time
the cache's live blocks move to the lowest ids (compact_blocks, copy_blocks).
Placing the new tokens (assign_slots) is measured elsewhere.
"""

import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # One request with four beams: latency counts.
        {"name": "beam_one", "op": "beam", "reqs": 1, "beams": 4, "vocab": 32000, "k": 4, "bf16": False, "eos": 2},
        # A decode step of a batch of requests, logits as the model's last product leaves them.
        {"name": "beam_decode", "op": "beam", "reqs": 32, "beams": 8, "vocab": 102400, "k": 8, "bf16": True,
         "eos": 2},
        # Many wide beams, twice as many candidates as beams, a vocabulary of odd size, fp32: the most work.
        {"name": "beam_wide", "op": "beam", "reqs": 64, "beams": 16, "vocab": 131071, "k": 32, "bf16": False,
         "eos": -1},
        # The block tables after a decode step of 32 requests with 8 beams each.
        {"name": "fork_beams", "op": "fork", "reqs": 32, "beams": 8, "ctx": 4096, "block": 16, "spare": 2, "ended": 0.0,
         "held": 0.0},
        # Many requests and long contexts; some requests end, and a prefix cache holds blocks of its own.
        {"name": "fork_large", "op": "fork", "reqs": 100, "beams": 8, "ctx": 16384, "block": 32, "spare": 2,
         "ended": 0.1, "held": 0.02},
        # A small pool after some requests have ended.
        {"name": "compact_small", "op": "compact", "reqs": 64, "beams": 1, "ctx": 2048, "block": 16, "spare": 2,
         "held": 0.0},
        # A large pool, half empty, with blocks that may not move.
        {"name": "compact_large", "op": "compact", "reqs": 500, "beams": 2, "ctx": 8192, "block": 32, "spare": 2,
         "held": 0.02},
        # The last blocks of forked beams: keys and values of 8 heads.
        {"name": "copy_fork", "op": "copy", "pairs": 192, "pad": 64, "block": 16, "widths": "1024,1024", "pool": 4096},
        # The moves of a compaction: latent vectors, index keys and their scales.
        {"name": "copy_compact", "op": "copy", "pairs": 8000, "pad": 1000, "block": 32, "widths": "576,128,1",
         "pool": 20000},
        # A few requests of moderate length: latency counts.
        {"name": "attend_small", "op": "attend", "reqs": 4, "each": 1, "ctx": 1000, "heads": 32, "kv": 8, "dim": 128,
         "block": 16, "window": 0, "e4m3": False},
        # A decode step of a full batch over ragged contexts: the most bytes.
        {"name": "attend_decode", "op": "attend", "reqs": 64, "each": 1, "ctx": 16384, "heads": 32, "kv": 8,
         "dim": 128, "block": 64, "window": 0, "e4m3": False},
        # Three very long requests, 8-bit cache, many query heads a key head.
        {"name": "attend_long", "op": "attend", "reqs": 3, "each": 1, "ctx": 131072, "heads": 64, "kv": 4, "dim": 128,
         "block": 32, "window": 0, "e4m3": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["beam", "fork", "compact", "copy", "attend", "attend"])
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        vocab = _log(rng, 65, 131072)
        reqs = _log(rng, 1, max(1, min(256, 64 * 16 * 131071 // (beams * vocab))))
        eos = rng.choice([-1, 0, 2, vocab - 1])
        k = min(rng.choice([1, beams, beams, 2 * beams, 50]), 63)
        return {"op": op, "reqs": reqs, "beams": beams, "vocab": vocab, "k": k, "bf16": rng.random() < 0.5,
                "eos": eos}
    if op in ("fork", "compact"):
        beams = rng.choice([1, 2, 4, 5, 8])
        block = rng.choice([1, 16, 24, 32, 64, 128])
        reqs = _log(rng, 1, 2000 // beams)
        ctx = _log(rng, 1, max(2, min(16384, 120000 * block // (reqs * beams))))
        case = {"op": op, "reqs": reqs, "beams": beams, "ctx": ctx, "block": block, "spare": rng.choice([1, 2, 3]),
                "held": rng.choice([0.0, 0.0, 0.05])}
        if op == "fork":
            case["ended"] = rng.choice([0.0, 0.1, 0.5])
        return case
    if op == "copy":
        block = rng.choice([1, 16, 24, 32, 64, 128])
        widths = rng.choice(["576", "576,128,1", "1024,1024", "72,72", "33,5"])
        row = sum(int(w) for w in widths.split(","))
        pairs = _log(rng, 1, min(20000, 8000 * 32 * 705 // (block * row)))
        return {"op": op, "pairs": pairs, "pad": rng.choice([0, 1, 100, 1000]), "block": block, "widths": widths,
                "pool": 2 * pairs + rng.choice([0, 7, 500])}
    kv, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 4, 5, 8, 8, 16, 20])
    dim = rng.choice([64, 128, 128, 128, 256])
    reqs, each = _log(rng, 1, 200), rng.choice([1, 1, 1, 2, 3])
    room = 64 * 16384 * 8 * 128 // (kv * dim * reqs * each * max(1, group // 4))
    ctx = _log(rng, 1, max(2, min(131072, room)))
    return {"op": op, "reqs": reqs, "each": each, "ctx": ctx, "heads": kv * group, "kv": kv, "dim": dim,
            "block": rng.choice([1, 16, 24, 32, 64, 128]), "window": rng.choice([0, 0, 0, 100, 1024]),
            "e4m3": rng.random() < 0.4}


# --------------------------------------------------------------------------- inputs

def _ints(g, lo, hi, n):
    """n whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int64)


def _lengths(g, ctx, n):
    """Lengths spread evenly from ctx down to half of it, in random order: ragged, with the same sum for every seed."""
    at = torch.arange(n, device=DEV) * (ctx - ctx // 2) // max(1, n - 1)
    return (ctx - at)[torch.randperm(n, generator=g, device=DEV)]


def _prepare_beam(c, g):
    rows = c["reqs"] * c["beams"]
    logits = torch.randn(rows, c["vocab"], generator=g, device=DEV).mul_(2.5)
    likely = torch.randint(0, c["vocab"], (rows, 8), generator=g, device=DEV)  # a few tokens stand out
    logits.scatter_add_(1, likely, torch.rand(rows, 8, generator=g, device=DEV) * 8)
    scores = -torch.rand(c["reqs"], c["beams"], generator=g, device=DEV) * 6
    return {"logits": logits.bfloat16() if c["bf16"] else logits, "scores": scores}


def _tables(c):
    """(columns, columns that the beams of a request share, blocks in use at most, blocks of the pool)"""
    cols = -(-c["ctx"] // c["block"]) + 1
    shared = c["ctx"] // 2 // c["block"] if c["beams"] > 1 else 0  # of the prompt: the shortest length has them
    need = c["reqs"] * (shared + c["beams"] * (cols - shared))
    return cols, shared, need, need * c["spare"]


def _prepare_tables(c, g):
    """Block tables of requests whose beams share the blocks of their prompt; some blocks are held elsewhere."""
    reqs, beams = c["reqs"], c["beams"]
    cols, shared, need, pool = _tables(c)
    ctx = _lengths(g, c["ctx"], reqs).repeat_interleave(beams)
    ids = torch.randperm(pool, generator=g, device=DEV)[:need].int()
    table = torch.empty(reqs * beams, cols, dtype=torch.int32, device=DEV)
    table[:, :shared] = ids[:reqs * shared].view(reqs, shared).repeat_interleave(beams, 0)
    table[:, shared:] = ids[reqs * shared:].view(reqs * beams, cols - shared)
    held = (torch.rand(pool, generator=g, device=DEV) < c["held"]) if c["held"] else None
    return {"table": table, "ctx": ctx.int(), "pool": pool, "held": held}


def _prepare_fork(c, g):
    s = _prepare_tables(c, g)
    rows = c["reqs"] * c["beams"]
    at = torch.arange(rows, device=DEV)
    parents = at // c["beams"] * c["beams"] + _ints(g, 0, c["beams"] - 1, rows)
    ended = torch.rand(c["reqs"], generator=g, device=DEV) < c["ended"]
    s["parents"] = torch.where(ended.repeat_interleave(c["beams"]), -1, parents).int()
    return s


def _prepare_copy(c, g):
    pool = c["pool"]
    picked = torch.randperm(pool, generator=g, device=DEV)[:2 * c["pairs"]].int().view(2, c["pairs"]).t()
    pairs = torch.full((c["pairs"] + c["pad"], 2), -1, dtype=torch.int32, device=DEV)
    pairs[:c["pairs"]] = picked
    caches = []
    for w in c["widths"].split(","):
        x = torch.randn(pool * c["block"], int(w), generator=g, device=DEV)
        caches.append(x.view(-1) if int(w) == 1 else x.bfloat16())  # scales a token, or vectors
    return {"pairs": pairs, "caches": caches}


def _prepare_attend(c, g):
    reqs, each = c["reqs"], c["each"]
    cols = -(-(c["ctx"] + each) // c["block"])
    cache_rows = reqs * cols * c["block"]
    ctx = _lengths(g, c["ctx"], reqs)

    def cache():
        x = torch.empty(cache_rows, c["kv"], c["dim"], dtype=torch.float8_e4m3fn if c["e4m3"] else torch.bfloat16,
                        device=DEV)
        for r in range(0, cache_rows, 1 << 17):
            part = x[r:r + (1 << 17)]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV))
        return x

    at = torch.arange(reqs * each, device=DEV)
    req = at // each
    scales = (torch.rand(2, c["kv"], generator=g, device=DEV) + 0.5) if c["e4m3"] else (None, None)
    return {"q": torch.randn(reqs * each, c["heads"], c["dim"], generator=g, device=DEV).bfloat16(),
            "k": cache(), "v": cache(), "ks": scales[0], "vs": scales[1], "req": req.int(),
            "ends": (ctx[req] + at % each).int(), "max_len": c["ctx"] + each, "scale": c["dim"] ** -0.5,
            "table": torch.randperm(reqs * cols, generator=g, device=DEV).int().view(reqs, cols)}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    make = {"beam": _prepare_beam, "fork": _prepare_fork, "compact": _prepare_tables, "copy": _prepare_copy,
            "attend": _prepare_attend}[case["op"]]
    return {"case": case, **make(case, g)}


# --------------------------------------------------------------------------- plain forms

def _plain_beam(s):
    c, scores = s["case"], s["scores"]
    reqs, beams, vocab = c["reqs"], c["beams"], c["vocab"]
    x = s["logits"].double()  # 64 bits: tokens of different beams are compared by sums of many terms
    m = x.amax(1, keepdim=True)
    lse = m + (x - m).exp_().sum(1, keepdim=True).log_()
    v = x.sub_(lse).view(reqs, beams, vocab).add_(scores.double()[:, :, None])
    ended = None
    if c["eos"] >= 0:
        ended = v[:, :, c["eos"]].float()
        v[:, :, c["eos"]] = -math.inf
    v = v.view(reqs, beams * vocab)
    at = torch.arange(beams * vocab, device=DEV)
    best, picked = [], []
    for _ in range(c["k"]):  # one after the other: equal values by ascending position
        top = v.amax(1, keepdim=True)
        first = torch.where(v == top, at, beams * vocab).amin(1, keepdim=True)
        best.append(top)
        picked.append(first)
        v.scatter_(1, first, -math.inf)
    best, picked = torch.cat(best, 1), torch.cat(picked, 1)
    none = best == -math.inf
    row = torch.arange(reqs, device=DEV)[:, None] * beams + picked // vocab
    out = {"scores": best.float(), "parents": torch.where(none, -1, row).int(),
           "tokens": torch.where(none, -1, picked % vocab).int()}
    if ended is not None:
        out["ended"] = ended
    return out


def _bits(ids, keep, pool):
    """Which of the pool's blocks occur among ids where keep is true."""
    mark = torch.zeros(pool + 1, dtype=torch.bool, device=DEV)
    mark[torch.where(keep, ids, pool).view(-1).long()] = True
    return mark[:pool]


def _ascending(mark, n):
    """The first n of the marked positions, in order, then -1."""
    out = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
    place = torch.where(mark, mark.cumsum(0) - 1, n).clamp(max=n)
    out[place] = torch.arange(mark.numel(), dtype=torch.int32, device=DEV)
    return out[:n]


def _plain_fork(s):
    b, pool, table = s["case"]["block"], s["pool"], s["table"]
    parents = s["parents"].long()
    rows, cols = parents.numel(), table.shape[1]
    live = parents >= 0
    p = parents.clamp(min=0)
    ctx = torch.where(live, s["ctx"].long()[p], 0)
    full, need = ctx // b, (ctx + b - 1) // b
    col = torch.arange(cols, device=DEV)[None]
    src = table[p]
    row = torch.arange(rows, device=DEV)
    first = torch.full((table.shape[0] + 1,), rows, device=DEV).scatter_reduce(
        0, torch.where(live, p, table.shape[0]), row, "amin")[p]
    partial = live & (need > full)
    last = src.gather(1, full[:, None].clamp(max=cols - 1)).squeeze(1).long()
    whole = _bits(src, col < full[:, None], pool)
    if s["held"] is not None:
        whole = whole | s["held"]
    lead = partial & (first == row)
    writers = torch.zeros(pool + 1, dtype=torch.int64, device=DEV).scatter_add(
        0, torch.where(lead, last, pool), torch.ones_like(last))[:pool]
    keeps = lead & ~whole[last] & (writers[last] == 1)
    taken = whole | (writers > 0)
    free = ~taken
    wants = partial & ~keeps
    order = wants.cumsum(0) - 1
    fresh = _ascending(free, rows)
    got = torch.where(wants, fresh[order.clamp(min=0)], -1)
    out = torch.where(col < need[:, None], src, -1)
    out = torch.where((col == full[:, None]) & wants[:, None], got[:, None], out)
    copies = torch.full((rows + 1, 2), -1, dtype=torch.int32, device=DEV)
    copies[torch.where(wants & (got >= 0), order, rows)] = torch.stack([last.int(), got], 1)
    copies[rows] = -1
    free = free & ~_bits(got, got >= 0, pool)
    return {"block_table": out, "ctx_lens": ctx.int(), "copies": copies[:rows],
            "free_blocks": _ascending(free, pool), "counts": torch.stack([free.sum(), wants.sum()]).int()}


def _plain_compact(s):
    b, pool, table = s["case"]["block"], s["pool"], s["table"]
    need = (s["ctx"].long() + b - 1) // b
    inside = torch.arange(table.shape[1], device=DEV)[None] < need[:, None]
    live = _bits(table, inside, pool)
    held = s["held"] if s["held"] is not None else torch.zeros(pool, dtype=torch.bool, device=DEV)
    moves_to = ~held
    movable = live & moves_to
    # The live blocks fit into the first places that may be used.
    below = moves_to & (moves_to.cumsum(0) <= movable.sum())
    most = pool // 2
    src, dst = _ascending(movable & ~below, most), _ascending(below & ~live, most)
    now = torch.arange(pool + 1, dtype=torch.int32, device=DEV)
    now[torch.where(src >= 0, src, pool).long()] = dst
    out = torch.where(inside, now[table.clamp(min=0).long()], -1)
    free = ~held & ~_bits(now[:pool], live, pool)
    return {"block_table": out, "moves": torch.stack([src, dst], 1), "free_blocks": _ascending(free, pool),
            "counts": torch.stack([free.sum(), (src >= 0).sum()]).int()}


def _plain_copy(s):
    pairs = s["pairs"][s["pairs"][:, 0] >= 0].long()
    for cache in s["caches"]:
        blocks = cache.view(s["case"]["pool"], -1)
        blocks[pairs[:, 1]] = blocks[pairs[:, 0]]
    return s["caches"]


def _plain_attend(s):
    c = s["case"]
    b, n, kv, dim = c["block"], s["max_len"], c["kv"], c["dim"]
    pos = torch.arange(n, device=DEV)
    end = s["ends"].long()[:, None]
    keep = pos[None] < end
    if c["window"]:
        keep &= pos[None] >= end - c["window"]
    out, lse = [], []
    for t0 in range(0, s["q"].shape[0], 16):  # some tokens at a time, for the memory's sake
        req = s["req"][t0:t0 + 16].long()
        cols = (pos // b).clamp(max=s["table"].shape[1] - 1)
        phys = s["table"][req][:, cols].long() * b + pos % b
        q = s["q"][t0:t0 + 16].float()
        tokens = q.shape[0]
        k = s["k"][phys].float().permute(0, 2, 3, 1).reshape(tokens * kv, dim, n)
        if s["ks"] is not None:
            k = (k.view(tokens, kv, dim, n) * s["ks"][:, None, None]).view(tokens * kv, dim, n)
        x = torch.bmm(q.view(tokens * kv, -1, dim), k).view(tokens, -1, n) * s["scale"]
        del k
        x = x.masked_fill_(~keep[t0:t0 + 16, None], -math.inf)
        m = x.amax(2, keepdim=True).clamp_(min=-3e38)
        p = (x - m).exp_()
        total = p.sum(2, keepdim=True)
        v = s["v"][phys].float().permute(0, 2, 1, 3).reshape(tokens * kv, n, dim)
        o = torch.bmm(p.view(tokens * kv, -1, n), v).view(tokens, kv, -1, dim)
        del v
        if s["vs"] is not None:
            o = o * s["vs"][:, None, None]
        out.append((o.view(tokens, -1, dim) / total.clamp(min=1e-38)).bfloat16())
        lse.append(torch.where(total > 0, m + total.log(), -math.inf).squeeze(2))
    return torch.cat(out), torch.cat(lse)


# --------------------------------------------------------------------------- one pass

def run(state):
    c, s = state["case"], state
    if own:
        import row_top_select_amd as rts
        if c["op"] == "beam":
            r = rts.beam_select(s["logits"], s["scores"], c["k"], eos=c["eos"])
            return {n: t for n, t in r._asdict().items() if t is not None}
        if c["op"] == "fork":
            return rts.fork_blocks(s["table"], s["ctx"], s["parents"], c["block"], s["pool"], held=s["held"])._asdict()
        if c["op"] == "compact":
            return rts.compact_blocks(s["table"], s["ctx"], c["block"], s["pool"], held=s["held"])._asdict()
        if c["op"] == "copy":
            rts.copy_blocks(s["caches"], s["pairs"], c["block"])
            return s["caches"]
        return rts.kv_attend_paged(s["q"], s["k"], s["v"], s["req"], s["ends"], s["table"], c["block"], s["scale"],
                                   k_scales=s["ks"], v_scales=s["vs"], window=c["window"], max_len=s["max_len"])
    plain = {"beam": _plain_beam, "fork": _plain_fork, "compact": _plain_compact, "copy": _plain_copy,
             "attend": _plain_attend}[c["op"]]
    return plain(s)


# --------------------------------------------------------------------------- floors

def work(case):
    """Each input once, each output once, and the products of the definition."""
    c = case
    if c["op"] == "beam":
        rows = c["reqs"] * c["beams"]
        return {"bytes": rows * (c["vocab"] * (2 if c["bf16"] else 4) + 8) + c["reqs"] * c["k"] * 12,
                "flops": rows * c["vocab"] * 4}
    if c["op"] in ("fork", "compact"):
        rows, (cols, _, _, pool) = c["reqs"] * c["beams"], _tables(c)
        lists = pool * 4 + (rows * 8 if c["op"] == "fork" else pool // 2 * 8) + (pool if c["held"] else 0)
        return {"bytes": rows * (cols * 7 + 8) + lists, "flops": 0}
    if c["op"] == "copy":
        row = sum(4 if w == "1" else 2 * int(w) for w in c["widths"].split(","))
        return {"bytes": 2 * c["pairs"] * c["block"] * row + (c["pairs"] + c["pad"]) * 8, "flops": 0}
    rows = c["reqs"] * c["each"]
    seen = c["ctx"] * 0.75
    if c["window"]:
        seen = min(seen, c["window"])
    per_key = 2 * c["kv"] * c["dim"] * (1 if c["e4m3"] else 2)
    return {"bytes": int(c["reqs"] * seen * per_key + rows * c["heads"] * (c["dim"] * 4 + 4)),
            "flops": int(rows * seen * c["heads"] * c["dim"] * 4)}


# --------------------------------------------------------------------------- 64 bits

def _exact_beam(c, s):
    scores, parents, tokens, ended = [], [], [], []
    for g in range(c["reqs"]):
        heaps = []
        for b in range(c["beams"]):
            row = s["logits"][g * c["beams"] + b].double()
            logp = row - torch.logsumexp(row, 0) + s["scores"][g, b].double()
            if c["eos"] >= 0:
                ended.append(logp[c["eos"]].clone())
                logp[c["eos"]] = -math.inf
            value, token = logp.topk(min(c["k"] + 1, c["vocab"]))
            heaps += [(-v, b, t) for v, t in zip(value.tolist(), token.tolist()) if v > -math.inf]
            # All tokens that tie with the last one take part.
            for t in torch.nonzero(logp == value[-1]).view(-1).tolist() if value[-1] > -math.inf else []:
                heaps.append((-float(value[-1]), b, t))
        heaps = sorted(set(heaps))[:c["k"]]
        heaps += [(math.inf, -1 - g * c["beams"], -1)] * (c["k"] - len(heaps))
        scores.append([-h[0] for h in heaps])
        parents.append([g * c["beams"] + h[1] for h in heaps])
        tokens.append([h[2] for h in heaps])
    out = {"scores": torch.tensor(scores, dtype=torch.float64, device=DEV),
           "parents": torch.tensor(parents, device=DEV), "tokens": torch.tensor(tokens, device=DEV)}
    if c["eos"] >= 0:
        out["ended"] = torch.stack(ended).view(c["reqs"], c["beams"])
    return out


def _exact_attend(c, s):
    group = c["heads"] // c["kv"]
    outs, sums = [], []
    for t in range(s["q"].shape[0]):
        end = int(s["ends"][t])
        p = torch.arange(max(0, end - c["window"]) if c["window"] else 0, end, device=DEV)
        page = s["table"][int(s["req"][t])].long()
        at = page[torch.div(p, c["block"], rounding_mode="floor")] * c["block"] + p.remainder(c["block"])
        k, v = s["k"][at], s["v"][at]
        for h in range(c["kv"]):
            q = s["q"][t, h * group:(h + 1) * group].double()
            factor = s["scale"] * (1.0 if s["ks"] is None else float(s["ks"][h]))
            z = (q @ k[:, h].double().t()) * factor
            lse = torch.logsumexp(z, 1)
            weight = torch.where(lse[:, None] == -math.inf, torch.zeros_like(z), torch.exp(z - lse[:, None]))
            o = weight @ v[:, h].double()
            outs.append(o if s["vs"] is None else o * s["vs"][h].double())
            sums.append(lse)
    rows = s["q"].shape[0]
    return torch.stack(outs).view(rows, c["heads"], c["dim"]), torch.stack(sums).view(rows, c["heads"])


def _exact_copy(c, s):
    source = torch.arange(c["pool"])
    for src, dst in s["pairs"].tolist():
        if src >= 0:
            source[dst] = src
    return [cache.double().view(c["pool"], -1)[source.to(DEV)].view(cache.shape) for cache in s["caches"]]


def exact(case, seed):
    if case["op"] == "beam":
        return _exact_beam(case, prepare(case, seed))
    if case["op"] == "attend":
        return _exact_attend(case, prepare(case, seed))
    if case["op"] == "copy":
        return _exact_copy(case, prepare(case, seed))
    return None  # whole numbers: the plain form's are the definition's
