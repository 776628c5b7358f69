"""kv_attend_paged: scores and scales at the ends of their range, split and whole."""

import math

import pytest

import beam_reference as ref
from gpu_common import say
from test_gpu_kv_attend import DEV, i32, plan, rts, setup  # noqa: F401 (rts: the fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** 127, -2.0 ** 127, 2.0 ** 120, 1e-30, 2.0 ** -126])
def test_scales_split(rts, scale):  # noqa: F811
    """Scores past the range of a 32-bit number: pieces are joined as one piece is, and give the value of the greatest score."""
    say("split scale", scale)
    assert plan(rts, 2, 4, 2, 64, 1 << 20)[0] > 1
    q, k, v, req, ends, table = setup(19, [700, 5000], 4, 2, 64, 16)
    got, lse = rts.kv_attend_paged(q.to(DEV), k.to(DEV), v.to(DEV), i32(req), i32(ends), i32(table), 16, scale,
                                   max_len=1 << 20)
    assert bool(torch.isfinite(got).all()) and not bool(torch.isnan(lse).any())
    for t in range(2):
        at = ref.seen_rows(table[req[t]], 0, ends[t], 16, 16, k.shape[0])
        for h in range(4):
            z = k[at, h // 2].double() @ q[t, h].double() * math.copysign(1.0, scale)
            if abs(scale) < 1:
                o, l, ob, lb = ref.kv_attend(q[t, h:h + 1], k[at, h // 2], v[at, h // 2], scale)
                assert bool(((got[t, h].cpu().double() - o[0]).abs() <= ob[0]).all())
                assert abs(float(lse[t, h]) - float(l[0])) <= float(lb[0])
                continue
            best, next_best = z.topk(2).values.tolist()
            if best - next_best > 64 * ref.U * float(z.abs().max()):
                assert torch.equal(got[t, h].cpu(), v[at[int(z.argmax())], h // 2])
            want = best * abs(scale)
            if want < 3e38:
                assert abs(float(lse[t, h]) / want - 1) < 1e-4
            else:
                assert float(lse[t, h]) == math.inf
    whole, whole_lse = rts.kv_attend_paged(q.to(DEV), k.to(DEV), v.to(DEV), i32(req), i32(ends), i32(table), 16, scale,
                                           workspace=None)
    if abs(scale) > 1:
        assert torch.equal(got, whole) and torch.equal(lse, whole_lse)


def test_scores_below_the_range(rts):  # noqa: F811
    """All scores below -3.4e38: the greatest has all of the weight, split and whole."""
    q, k, v, req, ends, table = setup(20, [5000], 2, 1, 64, 16)
    q, k = q.abs() + 1, k.abs() + 1
    args = (q.to(DEV), k.to(DEV), v.to(DEV), i32(req), i32(ends), i32(table), 16, -2.0 ** 125)
    for kw in ({"workspace": None}, {"max_len": 1 << 20}):
        got, lse = rts.kv_attend_paged(*args, **kw)
        assert (lse == -math.inf).all()
        at = ref.seen_rows(table[0], 0, 5000, 16, 16, k.shape[0])
        for h in range(2):
            z = -(k[at, 0].double() @ q[0, h].double())
            best, next_best = z.topk(2).values.tolist()
            assert best - next_best > 64 * ref.U * float(z.abs().max())
            assert torch.equal(got[0, h].cpu(), v[at[int(z.argmax())], 0])
