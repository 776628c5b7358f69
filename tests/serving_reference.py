"""Plain 64-bit implementations of the serving-path operators, written from
their definitions, and bounds on what 32-bit kernels may be off by.

U is one step of a 32-bit sum relative to its operands' magnitude: 2^-23, so
that a truncating adder is covered too.  A rounding to bf16 is off by at most
half a step, 2^-8 of the value."""

import math

import torch

U = 2.0 ** -23
BF16 = 2.0 ** -8


def slots(ctx, new, tokens, block, stride, free, table):
    """Lists in, dict of lists out; ``table`` (a list of lists) is extended in place."""
    starts, req, ends, where = [0], [], [], []
    used = 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(0, c), max(0, n)
        n = min(n, tokens - starts[-1])
        have, need = -(-c // block), -(-(c + n) // block)
        for b in range(have, need):
            if b < len(table[i]):
                table[i][b] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            b = p // block
            blk = table[i][b] if b < len(table[i]) else -1
            req.append(i)
            ends.append(p + 1)
            where.append(-1 if blk < 0 else blk * stride + p % block)
        starts.append(starts[-1] + n)
    pad = tokens - len(req)
    return {"query_starts": starts, "req_id": req + [-1] * pad, "row_ends": ends + [0] * pad,
            "slots": where + [-1] * pad, "used": [used], "block_table": table}


def phys(table_row, pos, block, stride, cache_rows):
    """Physical row of a position, or None."""
    b = pos // block
    if b >= len(table_row) or table_row[b] < 0:
        return None
    r = table_row[b] * stride + pos % block
    return r if r < cache_rows else None


def logits(q, keys, w, ks):
    """One token: q [heads, dim], keys [n, dim] (any float type), w [heads], ks [n] or None.
    Returns (logits [n], bound on a 32-bit result's error [n])."""
    q, keys, w = q.double(), keys.double(), w.double()
    heads, dim = q.shape
    x = torch.clamp(q @ keys.T, min=0)
    x = torch.where(torch.isnan(q @ keys.T), torch.full_like(x, math.nan), x)
    out = w @ x
    # dim steps in a dot product, then one for each head (of whole tiles of 32,
    # more than the kernels need: the heads that fill up a tile add none), one for
    # the halves' sum and one for the scale; every step relative to the sum of the
    # magnitudes.
    size = w.abs() @ (q.abs() @ keys.abs().T)
    bound = (dim + -(-heads // 32) * 32 + 2) * U * size
    if ks is not None:
        out, bound = out * ks.double(), bound * ks.double().abs()
    return out, bound


def attend(q, kv, scale, latent):
    """One token: q [heads, d], kv [n, d] the rows that it sees.
    Returns (out [heads, latent], lse [heads], bounds on both)."""
    q, kv = q.double(), kv.double()
    heads, d = q.shape
    n = kv.shape[0]
    if n == 0:
        return (q.new_zeros(heads, latent), q.new_full((heads,), -math.inf),
                q.new_zeros(heads, latent), q.new_zeros(heads))
    z = scale * (q @ kv.T)
    m = z.amax(1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(1, keepdim=True)
    v = kv[:, :latent]
    out = (p / total) @ v
    lse = (m + torch.log(total)).squeeze(1)
    # A score is off by d sums and the scale's two roundings; the exponent's
    # argument by a step of the score and of the maximum; exp2 by 2 steps.
    dz = (d + 2) * U * abs(scale) * (q.abs() @ kv.abs().T).amax(1) + 4 * U * z.abs().amax(1) + 2 * U
    size = (p / total) @ v.abs()
    # Relative: each weight by dz and its rounding to bf16, the weights' sum by
    # dz and n steps, the products' sum by n steps (and as many for rescaling
    # the running sums), the quotient by 2.  The result is rounded to bf16.
    rel = 2 * dz + BF16 + (3 * n + 4) * U
    out_bound = size * rel[:, None] * (1 + BF16) + out.abs() * BF16
    lse_bound = dz + (2 * n + 4) * U + 4 * U * lse.abs()
    return out, lse, out_bound, lse_bound


def merge(parts, lse):
    """parts [W, ..., dim], lse [W, ...]; returns (out, lse, bound on a 32-bit out, bound on lse)."""
    world = parts.shape[0]
    x = lse.double()
    m = x.amax(0).clamp(min=-1e300)
    w = torch.exp(x - m)
    total = w.sum(0)
    share = torch.where(w > 0, w / total.clamp(min=1e-300), torch.zeros_like(w))[..., None]
    v = torch.where(share > 0, parts.double(), torch.zeros_like(parts, dtype=torch.float64))
    out, size = (share * v).sum(0), (share * v.abs()).sum(0)
    # The exponent's argument is off by 2 steps of its own size and exp2 by 2;
    # both sums by world steps, the quotient by 2.
    gap = (m - x).where(w > 0, torch.zeros_like(x)).amax(0)
    rel = (2 * (2 * gap + 2) + 2 * world + 2) * U
    total_lse = torch.where(total > 0, m + torch.log(total.clamp(min=1e-300)), torch.full_like(total, -math.inf))
    finite = torch.where(torch.isinf(total_lse), torch.zeros_like(total_lse), total_lse)
    return out, total_lse, size * rel[..., None], rel + 4 * U * finite.abs()


def assert_close(got, want, bound, what):
    got, want, bound = got.double().cpu(), want.double().cpu(), bound.double().cpu()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~inf & ~torch.isnan(want)
    off = (got - want).abs()[ok]
    over = off > bound[ok]
    assert not bool(over.any()), (
        f"{what}: {int(over.sum())} of {over.numel()} values out of bounds, worst by "
        f"{float((off / bound[ok].clamp(min=1e-300)).max()):.3g} times the bound")
