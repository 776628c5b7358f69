"""Plain implementations of the operators of a beam-search step, written from their
definitions: the block calls on lists of whole numbers, the others in 64 bits with
bounds on what 32-bit kernels may be off by."""

import math

import torch

from serving_reference import BF16, U, phys

U24 = 2.0 ** -24  # half a step of a 32-bit number, relative to it


def beam_values(logits, score):
    """One beam: its tokens' values (64 bits), or None where it has no candidates, and a bound on the error of its lse."""
    x = logits.double()
    if not math.isfinite(score) or bool(torch.isnan(x).any()) or not math.isfinite(float(x.max())):
        return None, 0.0
    m = x.max()
    d = (x - m).clamp(min=-1e30)
    w = torch.exp(d)
    total = float(w.sum())
    # A term's exponent is off by half a step of the difference, of its product with log2(e) and of
    # that constant, exp2 by 2 steps; a wave's 8 terms are added to up to 64 chunks' sums, each of which may be
    # rescaled by a factor that is off like a term.
    each = 3 * U24 * float((w * d.abs()).sum()) / total + 2 * U
    bound = each + (8 + 64 * 4) * U + 3 * U24 * float(-d.min() if d.min() > -200 else 200.0)
    return score + ((x - m) - math.log(total)), bound


def check_beams(got, logits, scores, k, eos, what=""):
    """Checks a BeamStep: each beam's picks are the first of its own order, the order over the beams is that of the
    64-bit values (closer ones than twice the bound may change places), scores are the values."""
    groups, beams = scores.shape
    out_s, parents, tokens = got.scores.cpu(), got.parents.tolist(), got.tokens.tolist()
    vocab = logits.shape[1]
    for g in range(groups):
        values, orders, slack = {}, {}, 0.0
        for b in range(beams):
            v, bound = beam_values(logits[g * beams + b], float(scores[g, b]))
            slack = max(slack, bound)
            if v is None:
                if eos >= 0:
                    assert float(got.ended[g, b]) == -math.inf, f"{what}: group {g} beam {b} ended"
                continue
            if eos >= 0:
                want = float(v[eos])
                assert abs(float(got.ended[g, b]) - want) <= bound + U24 * abs(want) or float(got.ended[g, b]) == want, \
                    f"{what}: group {g} beam {b} ended {float(got.ended[g, b])} for {want}"
            x = logits[g * beams + b].double()
            order = torch.sort(x, descending=True, stable=True).indices[: k + 1].tolist()
            values[b] = v
            orders[b] = [t for t in order if t != eos and float(x[t]) > -math.inf][:k]
        best = sorted(((-float(values[b][t]), b, i) for b in values for i, t in enumerate(orders[b])))[:k]
        taken = dict.fromkeys(values, 0)
        last = math.inf
        for j in range(k):
            if j >= len(best):
                assert (parents[g][j], tokens[g][j], float(out_s[g, j])) == (-1, -1, -math.inf), f"{what}: tail {g}, {j}"
                continue
            b = parents[g][j] - g * beams
            assert b in values, f"{what}: group {g} place {j}: parent {parents[g][j]}"
            assert taken[b] < len(orders[b]) and tokens[g][j] == orders[b][taken[b]], (
                f"{what}: group {g} place {j}: beam {b} token {tokens[g][j]}, its next is "
                f"{orders[b][taken[b]] if taken[b] < len(orders[b]) else None}")
            taken[b] += 1
            v = float(values[b][tokens[g][j]])
            assert abs(v + best[j][0]) <= 2 * slack, f"{what}: group {g} place {j}: value {v} for {-best[j][0]}"
            assert v <= last + 2 * slack
            last = v
            assert abs(float(out_s[g, j]) - v) <= slack + U24 * abs(v), f"{what}: group {g} place {j}: score"


def _need(ctx, block, cols):
    ctx = max(0, ctx)
    return min(ctx // block, cols), min(-(-ctx // block), cols)


def fork(table, ctx, parents, block, pool, held, n_free):
    rows_in, cols = len(table), len(table[0]) if table else 0
    ok = lambda i: 0 <= i < pool  # noqa: E731
    alive = [p if 0 <= p < rows_in else None for p in parents]
    whole, lasts, named = set(), {}, set()
    for p in set(alive) - {None}:
        full, need = _need(ctx[p], block, cols)
        whole |= {i for i in table[p][:full] if ok(i)}
        named |= {i for i in table[p][:need] if ok(i)}
        if need > full and ok(table[p][full]):
            lasts.setdefault(table[p][full], set()).add(p)
    free = [i for i in range(pool) if i not in named and not (held and held[i])]
    out, lens, copies, wanted, seen = [], [], [], 0, set()
    for p in alive:
        row = [-1] * cols
        if p is not None:
            full, need = _need(ctx[p], block, cols)
            row[:need] = [i if ok(i) else -1 for i in table[p][:need]]
            if need > full and row[full] >= 0:
                i = row[full]
                if p in seen or i in whole or (held and held[i]) or len(lasts[i]) > 1:
                    row[full] = free[wanted] if wanted < len(free) else -1
                    if wanted < len(free):
                        copies.append([i, free[wanted]])
                    wanted += 1
            seen.add(p)
        out.append(row)
        lens.append(max(0, ctx[p]) if p is not None else 0)
    left = free[wanted:]
    return {"block_table": out, "ctx_lens": lens, "copies": copies + [[-1, -1]] * (len(parents) - len(copies)),
            "free_blocks": (left + [-1] * n_free)[:n_free], "counts": [len(left), wanted]}


def compact(table, ctx, block, pool, held, max_moves, n_free):
    cols = len(table[0]) if table else 0
    live = set()
    for row, c in zip(table, ctx):
        live |= {i for i in row[:_need(c, block, cols)[1]] if 0 <= i < pool}
    is_open = [not (held and held[i]) for i in range(pool)]
    movable = sorted(i for i in live if is_open[i])
    places = [i for i in range(pool) if is_open[i]][:len(movable)]
    bound = places[-1] + 1 if places else 0
    src = [i for i in movable if i >= bound]
    dst = [i for i in places if i not in live]
    assert len(src) == len(dst)
    moves = [[a, b] for a, b in zip(src, dst)][:max_moves]
    now = dict(map(tuple, moves))
    out = []
    for row, c in zip(table, ctx):
        need = _need(c, block, cols)[1]
        out.append([now.get(i, i) if 0 <= i < pool else -1 for i in row[:need]] + [-1] * (cols - need))
    after = {now.get(i, i) for i in live}
    free = [i for i in range(pool) if is_open[i] and i not in after]
    return {"block_table": out, "moves": moves + [[-1, -1]] * (max_moves - len(moves)),
            "free_blocks": (free + [-1] * n_free)[:n_free], "counts": [len(free), len(src)]}


def kv_attend(q, k, v, scale):
    """One token and key head: q [heads, dim], k and v [n, dim] what it sees.
    Returns (out [heads, dim], lse [heads], bounds on both)."""
    q, k, v = q.double(), k.double(), v.double()
    heads, dim = q.shape
    n = k.shape[0]
    if n == 0:
        zero = q.new_zeros(heads)
        return q.new_zeros(heads, dim), zero - math.inf, q.new_zeros(heads, dim), zero
    z = scale * (q @ k.T)
    m = z.amax(1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(1, keepdim=True)
    out = (p / total) @ v
    lse = (m + torch.log(total)).squeeze(1)
    # A score is off by dim sums and the scale's roundings (its product with a key scale among them); the
    # exponent's argument by a step of the score and of the maximum; exp2 by 2 steps.
    dz = (dim + 3) * U * abs(scale) * (q.abs() @ k.abs().T).amax(1) + 4 * U * z.abs().amax(1) + 2 * U
    size = (p / total) @ v.abs()
    # Relative: each weight by dz and what two bf16 terms leave of it, the weights' sum by dz and n steps, the
    # products' sum by 2 n steps (and as many for rescaling the running sums), the quotient and a value scale
    # by 4.  The result is rounded to bf16.
    rel = 2 * dz + BF16 * BF16 + (5 * n + 8) * U
    return (out, lse, size * rel[:, None] * (1 + BF16) + out.abs() * BF16,
            dz + (2 * n + 4) * U + 4 * U * lse.abs())


def seen_rows(table_row, begin, end, block, stride, cache_rows):
    rows = (phys(table_row, p, block, stride, cache_rows) for p in range(max(0, begin), min(end, len(table_row) * block)))
    return [r for r in rows if r is not None]
