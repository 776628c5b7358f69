"""The order of beam_select over beams, and how far its sums are off."""

import math

import pytest

from gpu_common import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 2.0 ** -24  # half a step of a 32-bit number, relative to it

# (groups, beams, vocab): one launch with four, two and one waves a row, and two launches
SHAPES = [(2, 4, 9000), (3, 7, 8000), (2, 16, 4000), (2, 20, 4000), (2, 4, 70001)]


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def lse_and_bound(x):
    """log sum e^x of a row (64 bits), and what a 32-bit sum of 2^(x log2 e - c) may be off by, c the whole number next to
    the maximum's product.  An exponent is rounded once, half a step of it, and log2 e has 0.23 half steps too little: 1.23 of
    |x - max| + 0.35.  An exponential is off by a step; the sum is taken relative to the maximum's own term, which has as
    much.  32 terms are added in 10 roundings, all that follows is in 64 bits."""
    x = x.double()
    m = x.max()
    w = torch.exp(x - m)
    total = float(w.sum())
    away = float((w * (m - x).clamp(max=1e6)).sum()) / total
    return float(m) + math.log(total), EPS * (1.23 * away + 2 * 0.35 + 4 + 10)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab", SHAPES)
@pytest.mark.parametrize("sharp", [0.3, 2.5, 8.0])
def test_sums(rts, dtype, groups, beams, vocab, sharp):
    """Every beam's best value alone: k = 1 and the other beams not in use."""
    say("sums", dtype, groups, beams, vocab, sharp)
    g = torch.Generator().manual_seed(vocab)
    logits = (torch.randn(groups * beams, vocab, generator=g) * sharp).to(dtype)
    x = logits.to(DEV)
    for b in range(beams):
        scores = torch.full((groups, beams), -math.inf)
        scores[:, b] = 0
        got = rts.beam_select(x, scores.to(DEV), 1)
        for i in range(groups):
            row = logits[i * beams + b]
            lse, bound = lse_and_bound(row)
            want = float(row.double().max()) - lse
            assert got.parents[i].tolist() == [i * beams + b]
            assert abs(float(got.scores[i, 0]) - want) <= bound + EPS * abs(want)
            assert float(got.scores[i, 0]) <= 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab", SHAPES)
def test_beams_a_little_apart_keep_their_order(rts, dtype, groups, beams, vocab):
    """Best values that differ by a few times what the sums may be off by, in any order of the beams."""
    say("a little apart", dtype, groups, beams, vocab)
    g = torch.Generator().manual_seed(vocab + 1)
    logits = (torch.randn(groups * beams, vocab, generator=g) * 2).to(dtype)
    scores = torch.empty(groups, beams)
    want = []
    for i in range(groups):
        place = torch.randperm(beams, generator=g).tolist()  # of each beam
        values, bounds = [], []
        for b in range(beams):
            row = logits[i * beams + b]
            lse, bound = lse_and_bound(row)
            best = float(row.double().max()) - lse
            scores[i, b] = -place[b] * 6e-6 - best
            values.append(float(scores[i, b]) + best)
            bounds.append(bound)
        order = sorted(range(beams), key=lambda b: -values[b])
        assert order == sorted(range(beams), key=lambda b: place[b])
        for a, b in zip(order, order[1:]):
            assert values[a] - values[b] > 2 * (bounds[a] + bounds[b])
        want.append([i * beams + b for b in order])
    got = rts.beam_select(logits.to(DEV), scores.to(DEV), beams)
    # The second best tokens lie further off than all of this (a bf16 row's may be equal to its best).
    top = logits.float().topk(2, 1).values
    assert float((top[:, 0] - top[:, 1]).min()) > 6e-6 * (beams + 1) or dtype == torch.bfloat16
    for i in range(groups):
        first = list(dict.fromkeys(got.parents[i].tolist()))
        assert first == want[i][:len(first)] and (len(first) == beams or dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab", [(2, 4, 1), (3, 16, 1), (1, 64, 1), (300, 3, 1), *SHAPES])
def test_certain_beams_go_by_their_number(rts, dtype, groups, beams, vocab):
    """One token that has all of the weight (a vocabulary of one, the others masked, or far below): its value is the beam's
    score to the last bit, whatever the logit, and equal beams go by their number."""
    say("certain", dtype, groups, beams, vocab)
    g = torch.Generator().manual_seed(beams)
    rows = groups * beams
    for others in (-math.inf, -1000.0) if vocab > 1 else (0.0,):
        logits = torch.full((rows, vocab), others)
        at = torch.randint(0, vocab, (rows,), generator=g)
        logits[torch.arange(rows), at] = torch.randn(rows, generator=g) * torch.tensor([1.0, 30.0, 0.01])[torch.arange(rows) % 3]
        if rows > 4 and vocab > 1:
            logits[1, at[1]], logits[2, at[2]], logits[3, at[3]] = 2.3, 7.7, -88.1
        logits = logits.to(dtype)
        k = min(beams, 64)
        for scores in (torch.zeros(groups, beams), torch.full((groups, beams), -3.7)):
            got = rts.beam_select(logits.to(DEV), scores.to(DEV), k)
            assert torch.equal(got.scores.cpu(), scores[:, :k])
            assert got.parents.cpu().tolist() == [[i * beams + b for b in range(k)] for i in range(groups)]
            assert got.tokens.cpu().tolist() == at.view(groups, beams)[:, :k].tolist()


@pytest.mark.parametrize("groups,beams,vocab", SHAPES)
def test_no_value_is_above_its_score(rts, groups, beams, vocab):
    """A probability is at most one."""
    say("at most one", groups, beams, vocab)
    g = torch.Generator().manual_seed(beams)
    for sharp, lift in ((5.0, 15.0), (1.0, 25.0), (40.0, 0.0)):
        logits = torch.randn(groups * beams, vocab, generator=g) * sharp
        logits[:, vocab // 2] += lift + torch.rand(groups * beams, generator=g) * 10
        got = rts.beam_select(logits.to(DEV), torch.zeros(groups, beams, device=DEV), beams)
        assert float(got.scores.max()) <= 0.0


@pytest.mark.parametrize("base", [1e5, -1e5, 9e5, -9e5])
def test_far_maxima_that_rise(rts, base):
    """Maxima that grow from group to group far from 0, where a product with log2 e has few digits behind its point."""
    say("far and rising", base)
    vocab = 40000
    row = base + torch.arange(vocab) // 400 * 0.125
    logits = torch.stack([row, row.flip(0), row[torch.randperm(vocab, generator=torch.Generator().manual_seed(0))]])
    got = rts.beam_select(logits.to(DEV), torch.zeros(3, 1, device=DEV), 1)
    for i in range(3):
        lse, bound = lse_and_bound(logits[i])
        want = float(logits[i].double().max()) - lse
        assert abs(float(got.scores[i, 0]) - want) <= bound + EPS * abs(want)
