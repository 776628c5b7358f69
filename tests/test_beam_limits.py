"""The largest calls of kv_attend_paged and beam_select: refused past the borders that the header names (on the CPU),
taken up to them."""

import ctypes
import math

import pytest

import beam_reference as ref
from serving_reference import assert_close
from test_beam_refusals import EUNSUP, attend, beam, lib

torch = pytest.importorskip("torch")

import row_top_select_amd as rts  # noqa: E402


def test_rows_of_attention():
    size, p = lib.kv_attend_paged_workspace_size, (ctypes.c_int64 * 2)()
    for rows, heads, kv in ((1 << 25, 1, 1), (1 << 22, 128, 8), (1 << 21, 16, 16), (1 << 20, 32 * 17, 16)):
        call = dict(rows=rows, heads=heads, kv=kv)
        over = rows * kv * -(-heads // kv // 16)
        assert over >= 1 << 25 and attend(**call) == EUNSUP, call
        plan = lambda n: lib.kv_attend_paged_plan(ctypes.c_int64(n), heads, kv, 128, 1, ctypes.c_int64(64), ctypes.c_int64(0), 1, p)  # noqa: E731
        assert plan(rows) == EUNSUP and size(rows, heads, kv, 128, 1, 64, 0) == 0
        assert plan((1 << 25) // (over // rows) - 1) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads,kv", [(131072, 128, 8), ((1 << 25) - 1, 1, 1)])
def test_most_rows_of_attention(rows, heads, kv):
    g = torch.Generator(device="cuda").manual_seed(rows)
    cache = [torch.randn(64, kv, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    q = torch.zeros(rows, heads, 64, dtype=torch.bfloat16, device="cuda")
    req = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    ends = torch.zeros(rows, dtype=torch.int32, device="cuda")
    some = [0, 1, 4097, rows // 2, rows - 2, rows - 1]
    q[some] = torch.randn(len(some), heads, 64, generator=g, device="cuda").bfloat16()
    req[some] = 0
    ends[some] = torch.tensor([64, 1, 33, 40, 7, 50], dtype=torch.int32, device="cuda")
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    out, lse = rts.kv_attend_paged(q, *cache, req, ends, table, 16, 0.125)
    k, v = (t.cpu() for t in cache)
    for t in some:
        at = ref.seen_rows([3, 0, 2, 1], 0, int(ends[t]), 16, 16, 64)
        for h in range(kv):
            mine = slice(h * heads // kv, (h + 1) * heads // kv)
            o, l, ob, lb = ref.kv_attend(q[t, mine].cpu(), k[at, h], v[at, h], 0.125)
            assert_close(out[t, mine], o, ob, f"out {t}")
            assert_close(lse[t, mine], l, lb, f"lse {t}")
    out[some] = 0
    lse[some] = -math.inf
    assert not bool(out.any()) and bool((lse == -math.inf).all())


def test_rows_of_a_selection():
    for groups, beams in ((1 << 24, 1), (1 << 18, 64), (5592406, 3)):
        assert beam(groups=groups, beams=beams, ld=100000) == EUNSUP
        assert lib.beam_select_workspace_size(0, groups, beams, 100000, 4) == 0
        assert lib.beam_select_workspace_size(0, groups - 1, beams, 100000, 4) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("groups,beams", [((1 << 24) - 1, 1), (4194304, 1), (5592405, 3), (262143, 64)])
def test_most_rows_of_a_selection(groups, beams):
    vocab = 3
    g = torch.Generator(device="cuda").manual_seed(groups)
    logits = torch.randn(groups * beams, vocab, generator=g, device="cuda")
    scores = -torch.rand(groups, beams, generator=g, device="cuda")
    got = rts.beam_select(logits, scores, 2)
    x = logits.double()
    v = (scores.double().view(-1, 1) + x - torch.logsumexp(x, 1, keepdim=True)).view(groups, beams * vocab)
    best, at = v.topk(2, 1)
    assert float((got.scores.double() - best).abs().max()) < 2e-6
    # Where the next values are further off than sums are, the picks are those of 64 bits.
    third = v.topk(3, 1).values if beams * vocab > 2 else None
    clear = (best[:, 0] - best[:, 1] > 4e-6) & (third[:, 1] - third[:, 2] > 4e-6)
    row = torch.arange(groups, device="cuda").view(-1, 1) * beams + at // vocab
    assert int(clear.sum()) > groups * 0.99
    assert torch.equal(got.parents[clear].long(), row[clear]) and torch.equal(got.tokens[clear].long(), (at % vocab)[clear])
