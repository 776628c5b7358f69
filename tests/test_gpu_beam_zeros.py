"""beam_select over logits of 0 and -0."""

import math

import pytest

from gpu_common import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab", [(1, 1, 2), (2, 4, 9000), (3, 7, 8000), (2, 16, 4000), (2, 20, 4000), (2, 4, 70001)])
def test_zeros_of_both_signs_are_equal(rts, dtype, groups, beams, vocab):
    """-0 and 0 are the same logit: the lower token comes first."""
    say("zeros", dtype, groups, beams, vocab)
    rows = groups * beams
    logits = torch.full((rows, vocab), -1.0)
    logits[:, ::2] = -0.0
    logits[:, 1::2] = 0.0
    if vocab > 2:
        logits[1:, :vocab // 3] = -2.0
        logits[1:, vocab // 3 + 1::5] = 0.0
    logits = logits.to(dtype)
    scores = torch.full((groups, beams), -math.inf)
    scores[:, 0] = 0.0
    for k in (1, 2, 9, 64):
        got = rts.beam_select(logits.to(DEV), scores.to(DEV), k)
        for i in range(groups):
            row = logits[i * beams].float()
            order = torch.sort(row, descending=True, stable=True).indices[:k].tolist()
            assert got.tokens[i].tolist()[:len(order)] == order
