"""beam_select against its definition in 64 bits."""

import math

import pytest

from beam_reference import check_beams
from gpu_common import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def inputs(seed, groups, beams, vocab, dtype, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(groups * beams, vocab, generator=g) * sharp).to(dtype)
    return logits, -torch.rand(groups, beams, generator=g) * 5


def run(rts, logits, scores, k, eos, pad=0, shift=0):
    rows, vocab = logits.shape
    wide = torch.full((rows, vocab + pad + shift), math.nan, dtype=logits.dtype, device=DEV)
    x = wide[:, shift:shift + vocab]
    x.copy_(logits)
    got = rts.beam_select(x, scores.to(DEV), k, eos=eos)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab,k,eos,pad,shift", [
    (1, 1, 1, 1, -1, 0, 0), (1, 1, 1, 1, 0, 0, 0), (1, 4, 65, 4, 2, 0, 0), (3, 5, 1000, 10, 999, 3, 1),
    (2, 8, 32000, 16, 7, 0, 0), (2, 3, 70001, 8, -1, 0, 3), (1, 2, 33000, 64, 5, 0, 0), (1, 64, 515, 64, -1, 5, 0),
    (5, 1, 20000, 63, 0, 0, 2), (300, 2, 2048, 2, 1, 0, 0), (1, 2, 200000, 7, -1, 1, 0), (1, 3, 512, 64, 511, 0, 0),
    (2, 2, 20, 50, 3, 0, 0), (2, 17, 6253, 32, 4, 0, 1), (3, 20, 70, 5, -1, 0, 0), (7, 4, 16384, 9, 1, 0, 0),
    (7, 4, 16385, 9, 1, 0, 0), (5, 8, 8192, 8, 0, 3, 0), (3, 16, 4096, 64, 9, 0, 5), (256, 2, 500, 4, 0, 0, 0), (2, 13, 7000, 26, -1, 0, 0),
    (2, 6, 300, 12, 7, 0, 0)])
def test_beam_select(rts, dtype, groups, beams, vocab, k, eos, pad, shift):
    say("beam", dtype, groups, beams, vocab, k, eos, pad, shift)
    logits, scores = inputs(vocab + k, groups, beams, vocab, dtype)
    check_beams(run(rts, logits, scores, k, eos, pad, shift), logits, scores, k, eos)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("values", [1, 2, 5])
@pytest.mark.parametrize("vocab", [700, 30001])
def test_ties_go_to_the_lowest_token(rts, dtype, values, vocab):
    say("ties", dtype, values, vocab)
    g = torch.Generator().manual_seed(values)
    logits = torch.randint(0, values, (6, vocab), generator=g).to(dtype)
    scores = torch.tensor([[0.0, -1.0, -0.25], [-3.0, 0.0, -0.5]])
    for k, eos in ((1, -1), (9, 0), (64, 3)):
        check_beams(run(rts, logits, scores, k, eos, shift=1), logits, scores, k, eos)


@pytest.mark.parametrize("vocab", [700, 32001])
def test_equal_beams_go_by_their_number(rts, vocab):
    """Rows of the same logits at every alignment: equal values to the last bit."""
    say("equal beams", vocab)
    row = torch.randn(1, vocab, generator=torch.Generator().manual_seed(1))
    for dtype in (torch.float32, torch.bfloat16):
        logits = row.to(dtype).expand(8, vocab)
        got = run(rts, logits, torch.zeros(1, 8), 24, -1, pad=0)
        check_beams(got, logits, torch.zeros(1, 8), 24, -1)
        x = logits[0].double()
        order = torch.sort(x, descending=True, stable=True).indices[:24].tolist()
        want = sorted((-float(x[t]), b, t) for t in order for b in range(8))[:24]
        assert got.parents[0].tolist() == [b for _, b, _ in want]
        assert got.tokens[0].tolist() == [t for _, _, t in want]


def test_ascending_rows(rts):
    """Every chunk holds larger logits than all before it, and the reverse."""
    up = torch.arange(40000, dtype=torch.float32).view(1, -1) / 1000
    logits = torch.cat([up, up.flip(1)])
    scores = torch.tensor([[0.0, -0.003]])
    for k in (1, 64):
        check_beams(run(rts, logits, scores, k, -1), logits, scores, k, -1)
    # one lane's elements hold all of the largest
    spread = torch.zeros(1, 32768)
    spread[0, 128::512] = torch.arange(64.0) + 1
    spread[0, 130::512] = torch.arange(64.0) + 1.5
    check_beams(run(rts, spread, torch.zeros(1, 1), 64, -1), spread, torch.zeros(1, 1), 64, -1)


def test_masked_logits_and_beams(rts):
    """-inf logits and scores are no candidates; few candidates leave tails."""
    logits, scores = inputs(3, 4, 4, 5000, torch.float32)
    logits[0, 10:] = -math.inf               # ten tokens
    logits[1] = -math.inf                    # none
    logits[2, 4999] = logits[2, 0] = math.inf
    logits[3, 77] = math.nan
    scores[1, 1:] = -math.inf                # a search's first step
    scores[2] = torch.tensor([math.nan, math.inf, -math.inf, -1.0])
    scores[3] = -math.inf
    logits[11, 5:] = -math.inf
    logits[11, 2] = -3.4028234663852886e38   # the lowest finite number is a candidate
    for eos in (-1, 3, 4999):
        check_beams(run(rts, logits, scores, 12, eos), logits, scores, 12, eos)
    got = run(rts, logits, scores, 12, 3)
    assert (got.parents[0, :9] == 0).all() and (got.parents[0, 9:] == -1).all()
    assert (got.parents[2, :4] == 11).all() and (got.parents[2, 4:] == -1).all()
    assert (got.parents[3] == -1).all() and (got.scores[3] == -math.inf).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["start", "end", "few", "rising", "falling", "tail of large ones"])
@pytest.mark.parametrize("beams,vocab", [(3, 6253), (3, 8200), (3, 70001), (7, 8000), (16, 4000), (17, 6253)])
def test_uneven_rows(rts, dtype, kind, beams, vocab):
    """Candidates in a few places of a row only, or all in its last elements."""
    say("uneven", dtype, kind, beams, vocab)
    logits, scores = inputs(vocab, 2, beams, vocab, torch.float32)
    if kind == "start":
        logits[:, 900:] = -math.inf
    elif kind == "end":
        logits[:, :-70] = -math.inf
    elif kind == "few":
        keep = torch.rand(logits.shape, generator=torch.Generator().manual_seed(2)) < 40 / vocab
        logits[~keep] = -math.inf
    elif kind == "rising":
        logits = logits.sort(dim=1).values
    elif kind == "falling":
        logits = logits.sort(dim=1, descending=True).values
    else:
        logits[:, -5:] += 30
    logits = logits.to(dtype)
    for k, eos in ((1, -1), (32, 0), (64, vocab - 1)):
        check_beams(run(rts, logits, scores, k, eos), logits, scores, k, eos)


def test_far_scores(rts):
    """Scores and logits at the ends of their range: the order is that of 64-bit values, then of the logits."""
    logits, scores = inputs(4, 1, 3, 900, torch.float32)
    scores[0] = torch.tensor([1e30, 1e30, -1e30])
    got = run(rts, logits, scores, 20, -1)
    first = torch.sort(logits[0], descending=True, stable=True).indices[:20].tolist()
    assert got.parents[0].tolist() == [0] * 20 and got.tokens[0].tolist() == first
    big = torch.full((1, 600), -3e38)
    big[0, 5], big[0, 9] = 3e38, 2e38
    got = run(rts, big, torch.zeros(1, 1), 2, -1)
    assert got.tokens[0].tolist() == [5, 9] and float(got.scores[0, 0]) == 0.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_far_logits(rts, dtype):
    """Logits at both ends of the range, whose maxima grow from group to group, and small ones behind them: the sums
    count what is equal to the largest, or near it."""
    vocab = 40000
    logits = torch.full((6, vocab), -math.inf)
    logits[0, ::10] = torch.arange(vocab // 10) * 1e33 - 3.2e38       # a new maximum every ten tokens
    logits[1, ::10] = torch.arange(vocab // 10) * 2e34 + 2.4e38
    logits[2, :30000], logits[2, 30000:] = -3e38, -2.5e38              # 10000 equal ones
    logits[3, :30000], logits[3, 30000:] = 2.5e38, 3e38
    logits[4, :20000], logits[4, 20000:] = -3.3e38, torch.randn(20000, generator=torch.Generator().manual_seed(0))
    logits[5, :20000], logits[5, 20000:39999] = 9e37, torch.randn(19999)
    logits = logits.to(dtype)
    scores = torch.zeros(6, 1)
    got = run(rts, logits, scores, 9, -1)
    check_beams(got, logits, scores, 9, -1)
    assert abs(float(got.scores[2, 0]) + math.log(10000)) < 1e-5 and abs(float(got.scores[3, 0]) + math.log(10000)) < 1e-5
    assert abs(float(got.scores[5, 0]) + math.log(20000)) < 1e-5


def test_logits_around_a_million(rts):
    """Maxima that cross the size at which the sums' terms change their form, upwards and from below."""
    vocab = 30000
    logits = torch.full((4, vocab), -math.inf)
    logits[0, :15000], logits[0, 15000:] = 999999.5, 1000000.5
    logits[1, :15000], logits[1, 15000:] = -1000000.5, -999999.5
    logits[2, :15000], logits[2, 15000:] = 1000000.5, 999999.5
    logits[3, :15000], logits[3, 15000:] = -999999.5, -1000000.5
    scores = torch.zeros(4, 1)
    got = run(rts, logits, scores, 5, -1)
    check_beams(got, logits, scores, 5, -1)
    want = -math.log(15000 * (1 + math.exp(-1)))
    assert (got.scores[:, 0].double() - want).abs().max() < 1e-5


@pytest.mark.parametrize("vocab", [9000, 90000])
def test_given_outputs_streams_and_replay(rts, vocab):
    logits, scores = inputs(5, 3, 4, vocab, torch.bfloat16)
    x, s = logits.to(DEV), scores.to(DEV)
    n = rts.beam_select_workspace_size(torch.bfloat16, 3, 4, vocab, 5)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = rts.BeamStep(torch.empty(3, 5, device=DEV), torch.empty(3, 5, dtype=torch.int32, device=DEV),
                       torch.empty(3, 5, dtype=torch.int32, device=DEV), torch.empty(3, 4, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rts.beam_select(x, s, 5, eos=1, out=out, workspace=ws, stream=side)
    side.synchronize()
    check_beams(out, logits, scores, 5, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rts.beam_select(x, s, 5, eos=1, out=out, workspace=ws)
    for seed in (6, 7, 8):
        logits, scores = inputs(seed, 3, 4, vocab, torch.bfloat16)
        x.copy_(logits)
        s.copy_(scores)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_beams(out, logits, scores, 5, 1)
        eager = rts.beam_select(x, s, 5, eos=1)
        assert all(torch.equal(a, b) for a, b in zip(eager, out))


@pytest.mark.parametrize("beams", [1, 5, 64])
def test_scores_in_place(rts, beams):
    logits, scores = inputs(beams, 7, beams, 3001, torch.float32)
    x, s = logits.to(DEV), scores.to(DEV)
    want = rts.beam_select(x, s, beams, eos=3)
    out = rts.BeamStep(s, torch.empty_like(want.parents), torch.empty_like(want.tokens), torch.empty_like(want.ended))
    rts.beam_select(x, s, beams, eos=3, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_far_rows(rts):
    """Rows past 2^32 bytes."""
    vocab, ld = 1000, 300_000_000
    flat = torch.empty(9 * ld + vocab, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((10, vocab), (ld, 1))
    logits, scores = inputs(9, 5, 2, vocab, torch.bfloat16)
    x.copy_(logits)
    check_beams(rts.beam_select(x, scores.to(DEV), 6, eos=0), logits, scores, 6, 0)


def test_no_groups(rts):
    got = rts.beam_select(torch.empty(0, 100, device=DEV), torch.empty(0, 4, device=DEV), 3, eos=1)
    assert got.scores.shape == (0, 3) and got.ended.shape == (0, 4)
