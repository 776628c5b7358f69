"""indexer_logits over the head counts that do not fill a matrix tile, and on the
paths that large calls take."""

import ctypes
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


def plan(rts, dtype, rows, heads, dim, cols, reqs=-1):
    """(tokens a workgroup, steps a workgroup, columns a step, stages of the key ring)."""
    p = (ctypes.c_int64 * 4)()
    code = rts.RTS_BF16 if dtype == torch.bfloat16 else rts.RTS_E4M3
    assert rts.raw_library().indexer_logits_plan(code, ctypes.c_int64(rows), heads, dim, ctypes.c_int64(cols),
                                                 ctypes.c_int64(reqs), p) == 0
    return list(p)


def scores(q, keys, w, ks):
    """ref.logits on the GPU with the bound of the real heads only."""
    x = q.double() @ keys.double().T
    out = w.double() @ torch.clamp(x, min=0)
    size = w.double().abs() @ (q.double().abs() @ keys.double().abs().T)
    bound = (q.shape[1] + q.shape[0] + 2) * ref.U * size
    return (out, bound) if ks is None else (out * ks.double(), bound * ks.double())


def check_row(got, want, bound, odt, what):
    if odt == torch.bfloat16:
        bound = bound * (1 + ref.BF16) + want.abs() * ref.BF16
    ref.assert_close(got, want, bound, what)


BF, E8 = DTYPES


@pytest.mark.parametrize("dtype,rows,heads,dim,cols,tokens,steps,stages", [
    (BF, 333, 32, 128, 8191, 11, 4, 1), (BF, 3, 32, 128, 150001, 3, 3, 2), (E8, 150, 128, 128, 9000, 2, 6, 1),
    (E8, 3, 32, 128, 400007, 3, 4, 1), (E8, 5, 32, 64, 300001, 5, 3, 2), (BF, 200, 128, 128, 5003, 2, 10, 1),
    (E8, 300, 64, 64, 9001, 11, 2, 1), (BF, 2, 64, 64, 200003, 2, 2, 2), (BF, 300, 24, 64, 6001, 15, 1, 1)])
def test_many_tokens_and_steps(rts, dtype, rows, heads, dim, cols, tokens, steps, stages):
    """Several tokens on one set of keys, with row ends before, inside and behind a workgroup's columns, and rings
    of keys over many steps, odd numbers of (token, head tile) items among them."""
    say("logits: workgroups of", tokens, "tokens and", steps, "steps", dtype, rows, heads, dim, cols)
    p = plan(rts, dtype, rows, heads, dim, cols)
    assert (p[0], p[1], p[3]) == (tokens, steps, stages), (p, "choose sizes that reach these paths again")
    g = gen(rows + cols)
    q = torch.randn(rows, heads, dim, generator=g).to(dtype).to(DEV)
    keys = torch.randn(cols, dim, generator=g).to(dtype).to(DEV)
    w = torch.randn(rows, heads, generator=g).to(DEV)
    ks = (torch.rand(cols, generator=g) + 0.5).to(DEV)
    ends = torch.randint(0, cols + 1, (rows,), generator=g).int()
    ends[::5] = torch.arange(cols, cols - len(ends[::5]), -1).int()
    ends[1] = 0
    ends[rows // 2] = cols + 7
    if rows > 4:
        ends[3], ends[4] = -2, p[1] * p[2]           # a span's end
    for odt, use_ks in ((torch.float32, True), (torch.bfloat16, False)):
        out = torch.full((rows, cols + 5), 77.0, dtype=odt, device=DEV)
        rts.indexer_logits(q, keys, w, key_scales=ks if use_ks else None, row_ends=ends.to(DEV), out=out)
        for t in range(rows):
            e = min(max(int(ends[t]), 0), cols)
            want, bound = scores(q[t], keys[:e], w[t], ks[:e] if use_ks else None)
            check_row(out[t, :e], want, bound, odt, f"row {t}")
            assert bool((out[t, e:] == 77.0).all()), "columns behind the row's end were written"
    again = torch.full_like(out, 77.0)
    rts.indexer_logits(q, keys, w, row_ends=ends.to(DEV), out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,counts,heads,dim,block,ctx,tokens,steps,stages", [
    (E8, [1] * 40 + [0] * 5, 64, 128, 64, 19000, 1, 8, 2), (BF, [1] * 40 + [0] * 5, 64, 128, 16, 19000, 1, 15, 2),
    (BF, [1] * 40 + [0] * 5, 40, 64, 16, 19000, 1, 8, 2), (E8, [1] * 40, 64, 128, 64, 19000, 2, 4, 1),
    (BF, [5, 1, 9, 0, 7, 5, 2, 11, 5, 3, 6, 4], 32, 128, 48, 19000, 5, 4, 1),
    (E8, [5, 1, 9, 0, 7, 5, 2, 11, 5, 3, 6, 4], 64, 64, 64, 29000, 5, 3, 2),
    (BF, [10, 9, 11, 30, 1, 0, 9, 10, 8], 64, 128, 1, 8500, 5, 3, 1),
    (E8, [15, 30, 1, 14] * 5, 32, 128, 128, 8800, 8, 3, 1)])
def test_paged_many_tokens_and_steps(rts, dtype, counts, heads, dim, block, ctx, tokens, steps, stages):
    """Several requests in one workgroup, tokens of none among them, missing pages in any step."""
    say("logits paged: workgroups of", tokens, "tokens and", steps, "steps", dtype, heads, dim, block, ctx)
    g = gen(sum(counts) + ctx)
    reqs = len(counts)
    req = [r for r, n in enumerate(counts) for _ in range(n)]
    lens = torch.randint(1, ctx, (reqs,), generator=g).tolist()
    lens[0], lens[1], lens[-1] = ctx, 3, ctx // 2 + 1
    ends = [lens[r] + sum(1 for x in req[:t] if x == r) + 1 for t, r in enumerate(req)]
    for at in (2, len(req) // 2, len(req)):            # tokens without a request, between others' too
        req.insert(at, -1 if at else reqs)
        ends.insert(at, 50)
    if len(req) > 8:
        ends[7] = 0
    rows = len(req)
    cols = ctx + max(counts) + 1
    p = plan(rts, dtype, rows, heads, dim, cols, reqs)
    assert (p[0], p[1], p[3]) == (tokens, steps, stages), (p, "choose sizes that reach these paths again")
    table_cols = -(-cols // block)
    stride = block + 1
    pages = min(reqs * table_cols, 1_500_000 // stride)  # requests may share pages
    table = torch.randint(0, pages, (reqs, table_cols), generator=g).int()
    table[torch.rand(table.shape, generator=g) < 0.03] = -1
    table[0, table_cols // 2] = pages + 3              # outside the cache
    cache_rows = pages * stride
    q = torch.randn(rows, heads, dim, generator=g).to(dtype).to(DEV)
    keys = torch.randn(cache_rows, dim, generator=g).to(dtype).to(DEV)
    w = torch.randn(rows, heads, generator=g).to(DEV)
    ks = (torch.rand(cache_rows, generator=g) + 0.5).to(DEV)
    td = table.to(DEV)
    req_d, ends_d = torch.tensor(req, dtype=torch.int32, device=DEV), torch.tensor(ends, dtype=torch.int32, device=DEV)
    for odt, use_ks in ((torch.float32, True), (torch.bfloat16, False)):
        out = torch.full((rows, cols + 3), 77.0, dtype=odt, device=DEV)
        rts.indexer_logits_paged(q, keys, w, req_d, ends_d, td, block, cols, key_scales=ks if use_ks else None,
                                 stride_rows=stride, out=out)
        for t in range(rows):
            e = ends[t] if 0 <= req[t] < reqs else 0
            pos = torch.arange(e, device=DEV)
            blk = td[max(req[t], 0)].long()[torch.div(pos, block, rounding_mode="floor")]
            at = blk * stride + pos % block
            there = (blk >= 0) & (at < cache_rows)
            at = torch.where(there, at, torch.zeros_like(at))
            want, bound = scores(q[t], keys[at], w[t], ks[at] if use_ks else None)
            want[~there] = math.nan
            check_row(out[t, :e], want, bound, odt, f"token {t} of request {req[t]}")
            assert bool((out[t, e:] == 77.0).all())
