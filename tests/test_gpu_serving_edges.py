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


def test_the_longest_contexts(rts):
    """Contexts of almost 2^31 positions, almost all on missing pages; a few tokens at the end of them."""
    say("latent paged: contexts of almost 2^31 tokens")
    block = 1 << 20
    cols = (1 << 31) // block
    table = torch.full((2, cols), -1, dtype=torch.int32)
    # Block 0 of a cache of 48 rows: positions 0..47 of a page.
    table[0, [0, 1000, cols - 2]] = 0
    table[1, [5, cols - 1]] = 0
    ctx = [(1 << 31) - 100 - 30, 3 * block + 7]
    q = torch.randn(5, 16, 576, generator=gen(12)).bfloat16()
    cache = torch.randn(48, 576, generator=gen(13)).bfloat16()
    out, lse = rts.latent_attend_paged(q.to(DEV), cache.to(DEV), i32([0, 3, 5]), i32(ctx), table.to(DEV), block, 0.07)
    for t in range(3):
        o, l, ob, lb = ref.attend(q[t], cache.repeat(3, 1), 0.07, 512)
        ref.assert_close(out[t], o, ob, f"out of token {t}")
        ref.assert_close(lse[t], l, lb, f"lse of token {t}")
    assert (out[3:] == 0).all() and (lse[3:] == -math.inf).all()   # page 5 lies behind the second request
    # The new tokens' own page, at the end of the range.
    table[0, cols - 1] = 0
    ctx[0] = (1 << 31) - block + 40
    out, lse = rts.latent_attend_paged(q.to(DEV), cache.to(DEV), i32([0, 3, 5]), i32(ctx), table.to(DEV), block, 0.07)
    for t in range(3):
        kv = torch.cat([cache.repeat(3, 1), cache[:41 + t]])
        o, l, ob, lb = ref.attend(q[t], kv, 0.07, 512)
        ref.assert_close(out[t], o, ob, f"out of token {t}")
        ref.assert_close(lse[t], l, lb, f"lse of token {t}")


def test_logits_of_the_longest_context(rts):
    """2^31 - 1 columns, almost all of them keys without a physical row."""
    say("logits paged: 2^31 - 1 columns")
    block, cols = 1 << 20, (1 << 31) - 1
    table = torch.full((1, (1 << 31) // block), -1, dtype=torch.int32)
    table[0, [0, 1000, -1]] = 0
    q = torch.randn(2, 8, 64, generator=gen(14)).bfloat16()
    keys = torch.randn(block, 64, generator=gen(15)).bfloat16()
    w = torch.randn(2, 8, generator=gen(16))
    out = torch.full((2, cols + 1), 77.0, dtype=torch.bfloat16, device=DEV)
    rts.indexer_logits_paged(q.to(DEV), keys.to(DEV), w.to(DEV), i32([0, 0]), i32([cols, cols - 70]), table.to(DEV), block,
                             cols, out=out)
    for t, end in ((0, cols), (1, cols - 70)):
        want, bound = ref.logits(q[t], keys, w[t], None)
        want, bound = want.to(DEV), (bound * (1 + ref.BF16) + want.abs() * ref.BF16).to(DEV)
        for page in (0, 1000, (1 << 31) // block - 1):
            n = min(block, end - page * block)
            ref.assert_close(out[t, page * block:page * block + n], want[:n], bound[:n], f"row {t}, page {page}")
        assert bool((out[t, end:] == 77.0).all())
        for a in range(0, end, 1 << 28):       # all other pages, a part at a time
            part = out[t, a:min(a + (1 << 28), end)].clone()
            for page in (0, 1000, (1 << 31) // block - 1):
                part[max(0, page * block - a):max(0, (page + 1) * block - a)] = math.nan
            assert bool(torch.isnan(part).all()), f"row {t}, columns from {a}"


@pytest.mark.parametrize("stride", [(1 << 33) + 3, (1 << 62) + 8, (1 << 63) - 1])
def test_slots_of_strides_past_32_bits(rts, stride):
    """A slot is the low 32 bits of id * stride + offset, whatever the stride is."""
    say("slots: a block stride of", stride)
    free = [5, (1 << 31) - 1, 1 << 20]
    m = rts.assign_slots(i32([0]), i32([9]), 9, torch.zeros(1, 3, dtype=torch.int32, device=DEV), i32(free), 3,
                         stride_rows=stride)
    low = [(free[t // 3] * stride + t % 3) & 0xFFFFFFFF for t in range(9)]
    assert m.slots.tolist() == [x - (1 << 32) if x >> 31 else x for x in low]
