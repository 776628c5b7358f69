"""indexer_logits over the head counts that do not fill a matrix tile, and on the
paths that large calls take."""

import math

import pytest

from gpu_common import say

torch = pytest.importorskip("torch")
import serving_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float8_e4m3fn]


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [1, 2, 5, 8, 31, 32, 33, 63, 97, 128])
def test_one_head_that_counts(rts, dtype, heads):
    """Every product is one exact number and only the last head has a weight: a logit is one product of 32-bit
    numbers, rounded once, whatever fills the head's tile."""
    say("logits: only the last head counts", dtype, heads)
    g = gen(heads)
    q = torch.zeros(3, heads, 128)
    q[:, :, 9] = 1.0
    keys = torch.randn(500, 128, generator=g).to(dtype)
    w = torch.zeros(3, heads)
    w[:, -1] = torch.tensor([0.7310585, -1.0 / 3.0, 1.1e-30])
    got = rts.indexer_logits(q.to(dtype).to(DEV), keys.to(DEV), w.to(DEV)).cpu()
    want = w[:, -1:] * torch.clamp(keys[:, 9].float(), min=0)[None]
    assert torch.equal(got, want)


@pytest.mark.parametrize("heads", [1, 7, 33, 64, 100])
def test_rounding_counts_the_heads_only(rts, heads):
    """The bound counts dim steps of a product's sum, one for each head, one for the halves' sum and one for
    the scale, and no more: heads that only fill a tile up add none."""
    say("logits: roundings of the real heads only", heads)
    g = gen(heads)
    q = torch.randn(4, heads, 64, generator=g).bfloat16()
    keys = torch.randn(700, 64, generator=g).bfloat16()
    w = torch.randn(4, heads, generator=g)
    got = rts.indexer_logits(q.to(DEV), keys.to(DEV), w.to(DEV))
    for t in range(4):
        want, _ = ref.logits(q[t], keys, w[t], None)
        size = w[t].double().abs() @ (q[t].double().abs() @ keys.double().abs().T)
        ref.assert_close(got[t], want, (64 + heads + 2) * ref.U * size, f"row {t}")


@pytest.mark.parametrize("weight", [1.0, -3e-20, 1e-30, -1e-44])
def test_infinities_with_any_weight(rts, weight):
    say("logits: a key's infinity under weights down to the smallest", weight)
    for heads in (1, 3, 32, 40):
        q = torch.rand(2, heads, 128, generator=gen(1)).bfloat16() + 0.5
        keys = torch.rand(70, 128, generator=gen(2)).bfloat16() + 0.5
        keys[33, 4], keys[50, 4] = math.inf, -math.inf
        w = torch.full((2, heads), weight)
        got = rts.indexer_logits(q.to(DEV), keys.to(DEV), w.to(DEV)).cpu()
        assert (got[:, 33] == math.copysign(math.inf, weight)).all() and (got[:, 50] == 0).all()
        rest = got[:, (torch.arange(70) != 33) & (torch.arange(70) != 50)]
        assert torch.isfinite(rest).all() and (torch.sign(rest) == math.copysign(1, weight)).all()
        zero = rts.indexer_logits(q.to(DEV), keys.to(DEV), torch.zeros(2, heads, device=DEV)).cpu()
        assert torch.isnan(zero[:, 33]).all() and (zero[:, :33] == 0).all()
