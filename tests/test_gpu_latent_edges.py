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
