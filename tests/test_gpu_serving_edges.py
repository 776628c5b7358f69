"""The operators around the select at the ends of their arguments' ranges."""

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


@pytest.mark.parametrize("stride,block", [(1 << 34, 1 << 30), ((1 << 62) + 8, 4), ((1 << 63) - 1, 2), (1 << 31, 1)])
def test_block_strides_past_the_cache(rts, stride, block):
    """block id * stride passes 64 bits: a physical row that does not exist, whatever its low bits are."""
    say("paged: a block stride of", stride)
    q = torch.randn(1, 8, 128, generator=gen(1)).bfloat16()
    keys = torch.randn(64, 128, generator=gen(2)).bfloat16()
    w = torch.randn(1, 8, generator=gen(3))
    table = i32([[0, block, 0]])
    got = rts.indexer_logits_paged(q.to(DEV), keys.to(DEV), w.to(DEV), i32([0]), i32([48]), table, 16, 48,
                                   stride_rows=stride).cpu()
    want, bound = ref.logits(q[0], keys[:16], w[0], None)
    ref.assert_close(got[0, :16], want, bound, "block 0")
    assert torch.isnan(got[0, 16:32]).all() and torch.equal(got[0, 32:], got[0, :16])
    lq = torch.randn(1, 16, 576, generator=gen(4)).bfloat16()
    cache = torch.randn(64, 576, generator=gen(5)).bfloat16()
    out, lse = rts.latent_attend_paged(lq.to(DEV), cache.to(DEV), i32([0, 1]), i32([47]), table, 16, 0.07,
                                       stride_rows=stride)
    o, l, ob, lb = ref.attend(lq[0], torch.cat([cache[:16], cache[:16]]), 0.07, 512)
    ref.assert_close(out[0], o, ob, "out")
    ref.assert_close(lse[0], l, lb, "lse")


def test_the_longest_list(rts):
    """2^31 - 1 entries, almost all -1; the few that are not lie at both ends and between."""
    say("latent rows: a list of 2^31 - 1 entries")
    k = (1 << 31) - 1
    ids = torch.full((1, k), -1, dtype=torch.int32, device=DEV)
    at = torch.tensor([0, 31, 32, 10 ** 9, k - 33, k - 2, k - 1], device=DEV)
    ids[0, at] = torch.arange(7, dtype=torch.int32, device=DEV)
    q = torch.randn(1, 16, 576, generator=gen(6)).bfloat16()
    cache = torch.randn(9, 576, generator=gen(7)).bfloat16()
    out, lse = rts.latent_attend_rows(q.to(DEV), cache.to(DEV), ids, 0.07)
    o, l, ob, lb = ref.attend(q[0], cache[:7], 0.07, 512)
    ref.assert_close(out[0], o, ob, "out")
    ref.assert_close(lse[0], l, lb, "lse")
    out, lse = rts.latent_attend_rows(q.to(DEV), cache.to(DEV), ids, 0.07, counts=i32([k - 1]))
    o, l, ob, lb = ref.attend(q[0], cache[:6], 0.07, 512)
    ref.assert_close(out[0], o, ob, "out of all but the last")


def test_numbers_that_do_not_fit_the_library_are_refused(rts):
    """A block size of 2^32 + 16 is not one of 16."""
    say("numbers past 32 and 64 bits")
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device=DEV)
    keys = torch.zeros(64, 128, dtype=torch.bfloat16, device=DEV)
    w, table = torch.zeros(1, 8, device=DEV), i32([[0, 1, 2]])
    lq = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(64, 576, dtype=torch.bfloat16, device=DEV)
    calls = [lambda b, s: rts.assign_slots(i32([3]), i32([2]), 4, table.clone(), i32([5, 6]), b, stride_rows=s),
             lambda b, s: rts.indexer_logits_paged(q, keys, w, i32([0]), i32([5]), table, b, 16, stride_rows=s),
             lambda b, s: rts.latent_attend_paged(lq, cache, i32([0, 1]), i32([5]), table, b, 0.1, stride_rows=s)]
    for call in calls:
        call(16, 16)
        for b, s in (((1 << 32) + 16, None), (16 - (1 << 32), None), (1 << 31, None), (16, (1 << 64) + 16), (16, 1 << 63)):
            with pytest.raises(ValueError, match="below"):
                call(b, s)
    with pytest.raises(ValueError, match="below"):
        rts.latent_attend_paged(lq, cache, i32([0, 1]), i32([5]), table, 16, 0.1, max_len=1 << 64)
    with pytest.raises(ValueError, match="below"):
        rts.indexer_logits_paged(q, keys, w, i32([0]), i32([5]), table, 16, 1 << 64)
    wide = torch.empty(0, 1 << 32, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="below"):
        rts.latent_attend_rows(lq[:0], cache, wide, 0.1)
    with pytest.raises(ValueError, match="below"):
        rts.assign_slots(i32([]), i32([]), 4, wide, i32([5, 6]), 16)
