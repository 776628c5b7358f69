"""Latent attention on the paths that large calls take: two and four groups of 32
query rows a workgroup, in one piece and in several, over listed rows and over
pages, with every mask.  The 64-bit reference runs on the GPU."""

import ctypes
import math

import pytest

from gpu_common import say

torch = pytest.importorskip("torch")
import serving_reference as ref  # noqa: E402
from test_gpu_latent_edges import attend_inf  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
i64 = ctypes.c_int64


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows_plan(rts, rows, heads, latent, k, split=True):
    """[groups of 32 query rows a workgroup, pieces]"""
    p = (ctypes.c_int32 * 2)()
    assert rts.raw_library().latent_attend_rows_plan(i64(rows), heads, latent, k, int(split), p) == 0
    return list(p)


def paged_plan(rts, tokens, reqs, heads, latent, max_len, split=True):
    p = (ctypes.c_int32 * 2)()
    assert rts.raw_library().latent_attend_paged_plan(i64(tokens), i64(reqs), heads, latent, i64(max_len),
                                                      int(split), p) == 0
    return list(p)


def check(out, lse, q, kv, scale, latent, what):
    """One token's results against its keys; slow where a key is not finite."""
    if bool(torch.isfinite(kv).all()):
        o, l, ob, lb = ref.attend(q, kv, scale, latent)
    else:
        o, l, ob, lb = attend_inf(q.cpu(), kv.cpu(), scale, latent)
    ref.assert_close(out, o, ob, f"out of {what}")
    ref.assert_close(lse, l, lb, f"lse of {what}")


@pytest.mark.parametrize("rows,heads,latent,k,groups,pieces", [
    (300, 128, 512, 100, 4, 1), (300, 130, 512, 100, 2, 1), (300, 64, 512, 100, 2, 1), (300, 100, 512, 70, 4, 1),
    (257, 60, 256, 300, 2, 1), (129, 128, 256, 400, 4, 1), (64, 128, 512, 2048, 4, 4), (40, 128, 512, 1500, 2, 3),
    (64, 100, 256, 900, 2, 2), (600, 50, 256, 70, 2, 1), (100, 100, 256, 1999, 4, 2)])
def test_rows_of_many_heads(rts, rows, heads, latent, k, groups, pieces):
    say("latent rows:", groups, "groups,", pieces, "pieces", rows, heads, latent, k)
    assert rows_plan(rts, rows, heads, latent, k) == [groups, pieces], "choose sizes that reach these paths again"
    g = gen(rows + heads + k)
    n = 5000
    q = torch.randn(rows, heads, latent + 64, generator=g).bfloat16()
    cache = torch.randn(n, latent + 64, generator=g).bfloat16()
    ids = torch.randint(0, n - 10, (rows, k), generator=g).int()
    counts = torch.randint(0, k + 1, (rows,), generator=g).int()
    counts[:8] = torch.tensor([k, 0, 1, 33, -4, k + 9, k, k // 2])
    cache[n - 10:] = math.nan                         # listed nowhere but behind counts and in row 6
    ids[2, 1:] = n - 5
    ids[3, 33:] = n - 5
    ids[0, 3:7], ids[0, 9], ids[0, 10] = -1, n, 2 ** 31 - 1
    ids[9] = -1                                       # nothing is left
    ids[10] = 17                                      # one row over and over
    ids[6, k // 2] = n - 7
    q[11] *= 30                                       # sharp scores: the maximum moves
    qd, cd, idd, nd = q.to(DEV), cache.to(DEV), ids.to(DEV), counts.to(DEV)
    for scale, workspace in ((192 ** -0.5, "auto"), (-0.07, None)):
        out, lse = rts.latent_attend_rows(qd, cd, idd, scale, d_latent=latent, counts=nd, workspace=workspace)
        for t in range(rows):
            at = idd[t, :min(max(int(counts[t]), 0), k)].long()
            at = at[(at >= 0) & (at < n)]
            check(out[t], lse[t], qd[t], cd[at], scale, latent, f"row {t}, {workspace}")
        assert torch.isnan(out[6]).all() and torch.isnan(lse[6]).all()


def paged_batch(seed, ctx, new, heads, latent, block, pad):
    g = gen(seed)
    reqs = len(ctx)
    cols = max(1, max(-(-(max(c, 0) + n) // block) for c, n in zip(ctx, new)))
    table = torch.randperm(reqs * cols, generator=g).int().view(reqs, cols)
    cache = torch.randn(reqs * cols * block, latent + 64, generator=g).bfloat16()
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = torch.randn(starts[-1] + pad, heads, latent + 64, generator=g).bfloat16()
    return q, cache, starts, table


def positions(ctx, new, j, mask):
    """What token j of a request sees; mask None: causal."""
    drafts = range(j + 1) if mask is None else [b for b in range(min(new, 64)) if mask >> b & 1]
    return [*range(max(ctx, 0)), *(max(ctx, 0) + b for b in drafts)]


def check_batch(rts, q, cache, starts, ctx, new, table, block, latent, tree, workspace, max_len=None):
    reqs = len(ctx)
    td = None
    if tree is not None:
        tree = tree + [0] * (q.shape[0] - len(tree))  # of padding tokens
        td = torch.tensor([x - (1 << 64) if x >> 63 else x for x in tree], dtype=torch.int64, device=DEV)
    out = torch.full((q.shape[0], q.shape[1], latent), 55.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 55.0, device=DEV)
    qd, cd = q.to(DEV), cache.to(DEV)
    rts.latent_attend_paged(qd, cd, i32(starts), i32(ctx), table.to(DEV), block, 0.07, d_latent=latent, tree=td,
                            out=out, lse=lse, workspace=workspace, max_len=max_len)
    for r in range(reqs):
        for t in range(starts[r], starts[r + 1]):
            pos = torch.tensor(positions(ctx[r], new[r], t - starts[r], None if tree is None else tree[t]),
                               dtype=torch.int64)
            b = torch.div(pos, block, rounding_mode="floor")
            pos, b = pos[b < table.shape[1]], b[b < table.shape[1]]
            blk = table[r].long()[b]
            at = blk * block + pos % block
            at = at[(blk >= 0) & (at < cache.shape[0])].to(DEV)
            check(out[t], lse[t], qd[t], cd[at], 0.07, latent, f"token {t} (request {r}), {workspace}")
    end = starts[-1]
    assert bool((out[end:] == 55.0).all()) and bool((lse[end:] == 55.0).all()), "rows behind the last token were written"
    return out, lse


def lengths(seed, reqs, tokens, longest):
    """Ragged cached and new lengths; requests without tokens and without a cache among them."""
    g = gen(seed)
    cut = torch.sort(torch.randint(0, tokens + 1, (reqs - 1,), generator=g)).values.tolist()
    new = [b - a for a, b in zip([0, *cut], [*cut, tokens])]
    ctx = [int(c) for c in torch.randint(0, longest, (reqs,), generator=g)]
    ctx[0], ctx[reqs // 2] = longest - new[0], 0
    return [max(c, 0) for c in ctx], new


@pytest.mark.parametrize("tokens,reqs,heads,latent,longest,block,groups,pieces", [
    (300, 100, 128, 512, 200, 16, 4, 1), (90, 30, 128, 512, 300, 48, 2, 1), (200, 3, 64, 512, 300, 64, 2, 1),
    (600, 2, 16, 512, 300, 32, 2, 1), (300, 60, 128, 256, 128, 1, 4, 1), (32, 32, 128, 512, 4000, 64, 4, 8),
    (16, 2, 128, 512, 3000, 64, 2, 14), (300, 4, 40, 256, 600, 16, 2, 1), (600, 9, 33, 256, 400, 64, 4, 1),
    (90, 30, 140, 512, 300, 48, 4, 1)])
@pytest.mark.parametrize("tree", [False, True])
def test_paged_of_many_heads(rts, tokens, reqs, heads, latent, longest, block, groups, pieces, tree):
    say("latent paged:", groups, "groups,", pieces, "pieces", tokens, reqs, heads, latent, longest, block, tree)
    pad = 2
    assert paged_plan(rts, tokens + pad, reqs, heads, latent, longest) == [groups, pieces], \
        "choose sizes that reach these paths again"
    ctx, new = lengths(tokens + heads, reqs, tokens, longest)
    q, cache, starts, table = paged_batch(tokens + heads, ctx, new, heads, latent, block, pad)
    masks = None
    if tree:
        g, masks = gen(9), []
        for n in new:
            mine = []
            for j in range(n):
                up = mine[int(torch.randint(0, j, (1,), generator=g))] if j else 0
                mine.append(up | (1 << j if j < 64 else 0))
            masks += mine
        masks[0], masks[-1] = 0, (1 << 64) - 1         # cached tokens only; drafts behind itself too
    for workspace in ("auto", None):
        check_batch(rts, q, cache, starts, ctx, new, table, block, latent, masks, workspace, longest)
    # Missing pages, a page outside the cache, a request with none, a table that ends early.
    if table.shape[1] > 2:
        table[0, 1] = -1
        table[-1, 0] = 10 ** 6
        table[reqs // 3] = -1
        check_batch(rts, q, cache, starts, ctx, new, table[:, :-1].contiguous(), block, latent, masks, "auto", longest)


@pytest.mark.parametrize("tokens,reqs,heads,latent,longest,groups,pieces", [
    (300, 100, 128, 512, 200, 4, 1), (90, 30, 128, 512, 300, 2, 1), (300, 60, 128, 256, 128, 4, 1),
    (300, 4, 40, 256, 600, 2, 1), (32, 32, 128, 512, 4000, 4, 14)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_paged_values_that_are_not_finite(rts, tokens, reqs, heads, latent, longest, groups, pieces, bad):
    """Every request's last new vector, one in its middle and everything behind the request: rows that do not see them
    are right, rows that do have their NaN."""
    say("latent paged: vectors that are not finite,", groups, "groups", tokens, reqs, heads, latent, longest, bad)
    assert paged_plan(rts, tokens, reqs, heads, latent, longest) == [groups, pieces], \
        "choose sizes that reach these paths again"
    block = 16
    ctx, new = lengths(tokens + heads + 1, reqs, tokens, longest)
    q, cache, starts, table = paged_batch(tokens + heads + 1, ctx, new, heads, latent, block, 0)

    def at(r, p):
        return int(table[r, p // block]) * block + p % block

    q[..., 7] = q[..., 7].abs() + 0.5                 # an infinity there has one sign a head
    q[:, ::2, 7] = -q[:, ::2, 7]
    for r in range(reqs):
        n = ctx[r] + new[r]
        for p in range(n, table.shape[1] * block):
            cache[at(r, p)] = bad
        if new[r] > 1 and r % 2 == 0:
            cache[at(r, n - 1)] = bad
        if new[r] > 2 and r % 3 == 0:
            cache[at(r, ctx[r] + new[r] // 2), 7] = bad
    for workspace in ("auto", None):
        check_batch(rts, q, cache, starts, ctx, new, table, block, latent, None, workspace, longest)
    tree = [1 << min(j, 63) for n in new for j in range(n)]
    check_batch(rts, q, cache, starts, ctx, new, table, block, latent, tree, "auto", longest)
