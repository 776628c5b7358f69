"""Latent attention at the edges of its inputs: scores at the ends of the 32-bit
range and values that are not finite, against the formulas in 64 bits."""

import math

import pytest

from gpu_common import say

torch = pytest.importorskip("torch")
import serving_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def both_forms(rts, q, cache, scale, latent=512, block=16, **kw):
    """The same attention of every row of q [rows, heads, d] over the whole cache [n, d]: over listed rows, and
    as one request a row over pages.  (The paged form's last key is its token's own.)"""
    rows, n = q.shape[0], cache.shape[0]
    ids = torch.arange(n, dtype=torch.int32).repeat(rows, 1).to(DEV)
    yield "rows", rts.latent_attend_rows(q.to(DEV), cache.to(DEV), ids, scale, d_latent=latent, **kw)
    cols = -(-n // block)
    table = torch.arange(cols, dtype=torch.int32).repeat(rows, 1).to(DEV)
    yield "paged", rts.latent_attend_paged(q.to(DEV), cache.to(DEV), i32(list(range(rows + 1))), i32([n - 1] * rows),
                                           table, block, scale, d_latent=latent, **kw)


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("power", [10, 24, 30, 34, 60, 100, 125])
def test_scores_of_any_size(rts, power, sign):
    """Every product is one exact number (all other elements of the queries are 0): sign * 1.5 * 2^(power + 1),
    for two keys the greatest by 2^-7 of it or more, which is beyond the range of an exponential from 2^20 on.  The result
    is then the mean of the two keys' values, and lse is their score + log 2."""
    say("latent: scores of 2 to the", power, sign)
    n = 200
    a = power // 2
    cache = torch.randn(n, 576, generator=gen(power))
    cache[:, 575] = 2.0 ** (power - a) * (1 if sign < 0 else 1 - 2.0 ** -7)
    cache[[3, 170], 575] = 2.0 ** (power - a) * (1 - 2.0 ** -7 if sign < 0 else 1)
    cache = cache.bfloat16()
    q = torch.zeros(1, 16, 576, dtype=torch.bfloat16)
    q[..., 575] = sign * 1.5 * 2.0 ** (a + 1)
    for scale in (1.0, 0.25, -0.25):
        qs = -q if scale < 0 else q
        for workspace in ("auto", None):
            for form, (out, lse) in both_forms(rts, qs, cache, scale, workspace=workspace):
                z = scale * qs[0, 0, 575].double() * cache[:, 575].double()
                p = torch.softmax(z, 0)
                want = p @ cache[:, :512].double()
                what = (form, scale, workspace)
                # The weights are exact or rounded once to bf16 (rows of equal scores), and so is the result.
                bound = 2 * ref.BF16 * (p @ cache[:, :512].double().abs()) + ref.BF16 * want.abs()
                ref.assert_close(out[0], want.expand(16, 512), bound.expand(16, 512), what)
                lse_want = torch.logsumexp(z, 0).expand(16)
                ref.assert_close(lse[0], lse_want, 4 * ref.U * (lse_want.abs() + 8), what)


def attend_inf(q, kv, scale, latent):
    """ref.attend of one token where some rows of kv are not finite: a score that is NaN or +inf makes the head
    NaN; one of -inf has the weight 0, which its values that are not finite turn into NaN."""
    z = scale * (q.double() @ kv.double().T)
    out, bound = torch.zeros(q.shape[0], latent, dtype=torch.float64), torch.zeros(q.shape[0], latent, dtype=torch.float64)
    lse, lse_bound = torch.full((q.shape[0],), -math.inf, dtype=torch.float64), torch.zeros(q.shape[0], dtype=torch.float64)
    for h in range(q.shape[0]):
        if bool((torch.isnan(z[h]) | (z[h] == math.inf)).any()):
            out[h], lse[h] = math.nan, math.nan
            continue
        none = z[h] == -math.inf
        o, l, ob, lb = ref.attend(q[h:h + 1], kv[~none], scale, latent)
        out[h], bound[h], lse[h], lse_bound[h] = o[0], ob[0], l[0], lb[0]
        out[h, (~torch.isfinite(kv[none][:, :latent])).any(0)] = math.nan
    return out, lse, bound, lse_bound


def check_seen(rts, seed, ctx, new, heads, latent, flaws, tree, block=16, all_low=False):
    """A paged batch where flaws: {(request, position): columns} of keys hold +inf, and every key too (column 0)
    with all_low; half of the heads have queries that turn them into -inf, the others into +inf."""
    g = gen(seed)
    reqs, tokens = len(ctx), sum(new)
    cols = -(-max(c + n for c, n in zip(ctx, new)) // block)
    table = torch.randperm(reqs * cols, generator=g).int().view(reqs, cols)
    cache = torch.randn(reqs * cols * block, latent + 64, generator=g).bfloat16()
    q = torch.randn(tokens, heads, latent + 64, generator=g).bfloat16()
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)

    def row(r, p):
        return int(table[r, p // block]) * block + p % block

    touched = sorted({c for cs in flaws.values() for c in cs} | ({0} if all_low else set()))
    low = torch.arange(heads) % 2 == 0
    for c in touched:
        q[:, low, c] = -q[:, low, c].abs() - 0.5
        q[:, ~low, c] = -q[:, ~low, c].abs() - 0.5 if all_low else q[:, ~low, c].abs() + 0.5
    for (r, p), cs in flaws.items():
        cache[row(r, p), cs] = math.inf
    if all_low:
        cache[:, 0] = math.inf
    td = None if tree is None else torch.tensor([x - (1 << 64) if x >> 63 else x for x in tree], device=DEV)
    results = []
    for workspace in ("auto", None):
        out, lse = rts.latent_attend_paged(q.to(DEV), cache.to(DEV), i32(starts), i32(ctx), table.to(DEV), block, 0.07,
                                           d_latent=latent, tree=td, workspace=workspace)
        out, lse = out.cpu(), lse.cpu()
        results.append((out, lse))
        for r in range(reqs):
            for t in range(starts[r], starts[r + 1]):
                j = t - starts[r]
                mine = range(j + 1) if tree is None else [b for b in range(min(new[r], 64)) if tree[t] >> b & 1]
                at = torch.tensor([row(r, p) for p in [*range(ctx[r]), *(ctx[r] + b for b in mine)]], dtype=torch.int64)
                o, l, ob, lb = attend_inf(q[t], cache[at], 0.07, latent)
                ref.assert_close(out[t], o, ob, f"out of token {t} (request {r}), {workspace}")
                ref.assert_close(lse[t], l, lb, f"lse of token {t} (request {r}), {workspace}")
    return results


FLAWS = {(0, 3): [5], (0, 72): [0, 63, 64], (0, 74): [130, 255], (1, 2): [9], (1, 3): [9, 31]}


@pytest.mark.parametrize("latent", [512, 256])
@pytest.mark.parametrize("heads", [1, 2, 16, 70, 128])
def test_seen_infinities(rts, heads, latent):
    """Keys with infinities in stages where rows see different keys and in others: every row that sees one has its
    NaN, every row that does not has none."""
    say("latent paged: infinities that are seen", heads, latent)
    ctx, new = [70, 0, 300], [6, 5, 2]
    check_seen(rts, heads, ctx, new, heads, latent, {**FLAWS, (2, 301): [7], (2, 130): [200]}, None)
    tree = [1 << j | (1 << (j // 2)) for n in new for j in range(n)]
    tree[1] = 0
    check_seen(rts, heads + 1, ctx, new, heads, latent, {**FLAWS, (2, 301): [7]}, tree)


@pytest.mark.parametrize("heads", [16, 128])
def test_seen_infinities_in_many_stages(rts, heads):
    """More drafted tokens than a stage has keys: several stages with masks, flaws in each."""
    say("latent paged: infinities in several masked stages", heads)
    flaws = {(0, p): [p % 512, 511 - p % 100] for p in range(20, 130, 7)}
    check_seen(rts, 7, [40], [100], heads, 512, flaws, None)


@pytest.mark.parametrize("latent", [512, 256])
def test_all_scores_minus_infinity(rts, latent):
    """Every key's score is -inf: weights 0, lse -inf, NaN where the values are not finite; in one piece and in
    several alike, and over listed rows too."""
    say("latent: all scores -inf", latent)
    a, b = check_seen(rts, 3, [900, 10, 0], [2, 3, 1], 16, latent, {}, None, all_low=True)
    for x, y in zip(a, b):
        assert torch.equal(torch.isnan(x), torch.isnan(y))
    assert torch.isnan(a[0][..., 0]).all() and (a[0][..., 1:] == 0).all() and (a[1] == -math.inf).all()
    q = -torch.rand(2, 16, latent + 64, generator=gen(4)).bfloat16() - 0.5
    cache = torch.randn(700, latent + 64, generator=gen(5)).bfloat16()
    cache[:, 2] = math.inf
    cache[600:, 2] = 1.0
    ids = torch.arange(600).int().repeat(2, 1)
    for extra in (0, 40):                        # all of weight 0; some ordinary keys behind them
        ids2 = torch.cat([ids, 600 + torch.arange(extra).int().repeat(2, 1)], 1)
        for workspace in ("auto", None):
            out, lse = rts.latent_attend_rows(q.to(DEV), cache.to(DEV), ids2.to(DEV), 0.07, d_latent=latent,
                                              workspace=workspace)
            for t in range(2):
                o, l, ob, lb = attend_inf(q[t], cache[ids2[t].long()], 0.07, latent)
                ref.assert_close(out[t], o, ob, f"out {t} {extra} {workspace}")
                ref.assert_close(lse[t], l, lb, f"lse {t} {extra} {workspace}")


@pytest.mark.parametrize("scale,power", [(2.0 ** 127, -60), (-(2.0 ** 127), -60), (1e-38, 0), (-3e-39, 0), (1e-45, 0),
                                         (1e-36, 50)])
def test_scales_at_the_ends(rts, scale, power):
    """Scales from the largest that is taken to the smallest there is; queries and keys make up for them."""
    say("latent: a scale of", scale)
    n = 300
    q = (torch.randn(1, 16, 576, generator=gen(8)) * 2.0 ** power).bfloat16()
    cache = torch.randn(n, 576, generator=gen(9)).bfloat16()
    cache[:, 512:] = (cache[:, 512:].float() * 2.0 ** power).bfloat16()
    q[..., :512] = 0                                     # the scores come from the positional part
    scale32 = float(torch.tensor(scale, dtype=torch.float32))
    for workspace in ("auto", None):
        for form, (out, lse) in both_forms(rts, q, cache, scale, workspace=workspace):
            o, l, ob, lb = ref.attend(q[0], cache, scale32, 512)
            ref.assert_close(out[0], o, ob, (form, workspace))
            ref.assert_close(lse[0], l, lb, (form, workspace))


@pytest.mark.parametrize("latent", [512, 256])
def test_scale_zero(rts, latent):
    """0 times a product: the mean of the values; NaN where the product is not finite, whichever side it comes from."""
    say("latent: a scale of 0")
    n = 150
    q = torch.randn(1, 16, latent + 64, generator=gen(10)).bfloat16()
    cache = torch.randn(n, latent + 64, generator=gen(11)).bfloat16()
    q[0, 3, latent + 5], q[0, 8, 2], q[0, 15, 0] = math.nan, math.inf, -math.inf
    for scale in (0.0, -0.0):
        for form, (out, lse) in both_forms(rts, q, cache, scale, latent):
            bad = torch.zeros(16, dtype=torch.bool)
            bad[[3, 8, 15]] = True
            assert torch.isnan(out[0, bad]).all() and torch.isnan(lse[0, bad]).all(), form
            o, l, ob, lb = ref.attend(q[0, ~bad], cache, 0.0, latent)
            ref.assert_close(out[0, ~bad], o, ob, form)
            ref.assert_close(lse[0, ~bad], l, lb, form)
    cache[70, latent + 1] = math.inf
    for form, (out, lse) in both_forms(rts, q, cache, 0.0, latent):
        assert torch.isnan(out).all() and torch.isnan(lse).all(), form
