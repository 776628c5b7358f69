"""Latent attention with scales that carry scores past the range of 32 bits, split and whole."""

import math

import pytest

import serving_reference as ref
from gpu_common import say
from test_gpu_latent_edges import both_forms, gen, rts  # noqa: F401 (rts: the fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("scale", [2.0 ** 127, -2.0 ** 127, 2.0 ** 100, 3.0, 1.0, 0.75])
def test_scores_past_the_range(rts, scale, sign, heads):  # noqa: F811
    """Every product is one exact number; two keys, far from each other, have the greatest, by 2^24 and more after the
    scale.  The result is the mean of their values, lse their score + log 2 (infinite past 3.4e38), however the keys are cut."""
    say("latent scale", scale, sign, heads)
    n = 4000
    cache = torch.randn(n, 576, generator=gen(heads))
    up = (sign > 0) == (scale > 0)
    size = 2.0 ** 30 if abs(scale) < 4 else 2.0 ** 4
    cache[:, 575] = size * (1 - 2.0 ** -6 if up else 1)
    cache[[3, 3900], 575] = size * (1 if up else 1 - 2.0 ** -6)
    cache = cache.bfloat16()
    q = torch.zeros(1, heads, 576, dtype=torch.bfloat16)
    q[..., 575] = sign * 1.5
    want = cache[[3, 3900], :512].double().mean(0)
    bound = ref.BF16 * want.abs() + 2 * ref.BF16 * cache[[3, 3900], :512].double().abs().mean(0)
    best = scale * sign * 1.5 * float(cache[3, 575].double())
    for workspace in ("auto", None):
        for form, (out, lse) in both_forms(rts, q, cache, scale, workspace=workspace):
            what = (form, scale, workspace)
            ref.assert_close(out[0], want.expand(heads, 512), bound.expand(heads, 512), what)
            if abs(best) > 3.5e38:
                assert (lse == math.copysign(math.inf, best)).all(), what
            else:
                assert float((lse.double() / (best + math.log(2)) - 1).abs().max()) < 4 * ref.U, what
