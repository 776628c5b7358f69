"""The serving-path operators around the select against plain 64-bit
implementations: slot maps, indexer logits, latent attention over selected rows
and over paged caches, and the join of ranks' partial results."""

import math

import numpy as np
import pytest

from gpu_common import assert_ids_equal, host, say

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


# ------------------------------------------------------------------ slot maps

def check_slots(rts, ctx, new, tokens, block, stride, free, cols, extra_cols=0, out=None):
    rng = np.random.default_rng(len(ctx) + tokens)
    wide = rng.integers(0, 1000, size=(len(ctx), cols + extra_cols)).astype(np.int32)
    t = torch.from_numpy(wide.copy()).to(DEV)
    view = t[:, :cols]
    got = rts.assign_slots(i32(ctx), i32(new), tokens, view, i32(free), block, stride_rows=stride, out=out)
    want = ref.slots(ctx, new, tokens, block, stride, free, wide[:, :cols].tolist())
    for name in rts.SlotMap._fields:
        assert_ids_equal(host(getattr(got, name))[None], np.array([want[name]], np.int64).astype(np.int32), name)
    assert np.array_equal(host(view), np.array(want["block_table"], np.int32).reshape(len(ctx), cols))
    if extra_cols:
        assert np.array_equal(host(t)[:, cols:], wide[:, cols:]), "columns behind the table changed"
    return got


@pytest.mark.parametrize("reqs,new,block,pad", [(1, 1, 64, 0), (64, 1, 64, 0), (7, 33, 16, 5), (300, 40, 1, 100),
                                                (1000, 3, 48, 0), (8192, 2, 16, 7), (5, 700, 32, 0)])
def test_assign_slots(rts, reqs, new, block, pad):
    say("slots", reqs, new, block, pad)
    rng = np.random.default_rng(reqs + new)
    ctx = rng.integers(0, 200, size=reqs).tolist()
    lens = rng.integers(0, new + 1, size=reqs).tolist()
    ctx[0] = 0
    cols = -(-(200 + new) // block)
    free = rng.permutation(reqs * cols + 10)[: reqs * (new // block + 2)].tolist()
    check_slots(rts, ctx, lens, sum(lens) + pad, block, block, free, cols, extra_cols=3)


def test_assign_slots_edges(rts):
    say("slots edges")
    check_slots(rts, [], [], 4, 16, 16, [3], 2)                                    # no requests: only padding
    check_slots(rts, [5, 0], [0, 0], 0, 16, 16, [], 2)                             # no tokens
    check_slots(rts, [5, 0, 9], [0, 0, 0], 3, 16, 16, [1], 2)                      # nothing new
    check_slots(rts, [-3, 8], [2, -9], 6, 4, 4, [7, 6], 4)                         # negative lengths
    check_slots(rts, [0, 16, 31], [40, 16, 2], 58, 16, 24, [9, 8], 4)              # the free list runs out
    check_slots(rts, [0, 16, 31], [40, 16, 2], 58, 16, 16, list(range(20)), 2)     # past the table
    check_slots(rts, [3, 3, 3], [10, 10, 10], 17, 8, 8, list(range(20)), 4)        # cut at the capacity
    check_slots(rts, [0], [3], 3, 1 << 20, (1 << 20) + 7, [4000], 1)               # a row past 2^31: low 32 bits
    check_slots(rts, [0], [5000], 5000, 3, 3, list(range(2000)), 1700)             # no power of two


def test_assign_slots_given_outputs_and_replay(rts):
    say("slots: given outputs, graph replay")
    reqs, tokens = 3, 12
    out = rts.SlotMap(*(torch.full((n,), -7, dtype=torch.int32, device=DEV) for n in (reqs + 1, tokens, tokens,
                                                                                    tokens, 1)))
    ctx, new = i32([0, 4, 9]), i32([1, 2, 3])
    table, free = torch.full((3, 4), -1, dtype=torch.int32, device=DEV), i32(list(range(50, 70)))
    rts.assign_slots(ctx, new, tokens, table, free, 4, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rts.assign_slots(ctx, new, tokens, table, free, 4, out=out)
    for c, n in (([0, 4, 9], [1, 2, 3]), ([3, 0, 8], [4, 4, 4]), ([1, 1, 1], [0, 11, 0])):
        ctx.copy_(i32(c))
        new.copy_(i32(n))
        table.fill_(77)
        g.replay()
        want = ref.slots(c, n, tokens, 4, 4, list(range(50, 70)), [[77] * 4 for _ in range(3)])
        for name in rts.SlotMap._fields:
            assert host(getattr(out, name)).tolist() == want[name], name
        assert host(table).tolist() == want["block_table"]


# ------------------------------------------------------------- indexer logits

def index_inputs(seed, rows, heads, dim, n_keys, dtype, pad=0):
    g = gen(seed)
    q = torch.randn(rows, heads * dim + pad, generator=g).to(dtype)[:, :heads * dim]
    keys = torch.randn(n_keys, dim + pad, generator=g).to(dtype)[:, :dim]
    w = torch.randn(rows, heads + 3, generator=g)[:, :heads]
    ks = torch.rand(n_keys, generator=g) + 0.5
    return q, keys, w, ks


def on_dev(t, pad):
    """A copy on the GPU with the same padded row stride."""
    if not pad:
        return t.contiguous().to(DEV)
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t.to(DEV)
    return wide[:, :t.shape[1]]


DTYPES = [torch.bfloat16, torch.float8_e4m3fn]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows,heads,dim,cols,pad", [(1, 1, 128, 1, 0), (3, 32, 128, 64, 0), (5, 33, 64, 65, 16),
                                                    (9, 64, 128, 300, 32), (2, 128, 128, 257, 0),
                                                    (40, 7, 64, 31, 0), (17, 64, 64, 1030, 16)])
def test_indexer_logits(rts, dtype, rows, heads, dim, cols, pad):
    say("logits", dtype, rows, heads, dim, cols, pad)
    q, keys, w, ks = index_inputs(rows + cols, rows, heads, dim, cols, dtype, pad)
    ends = torch.randint(0, cols + 1, (rows,), generator=gen(rows)).int()
    ends[0] = cols
    if rows > 2:
        ends[1], ends[2] = 0, cols + 5  # an empty row; past the columns: clamped
    for use_ks, use_ends, odt in ((False, False, torch.float32), (True, True, torch.float32),
                                  (True, True, torch.bfloat16)):
        out = torch.full((rows, cols + 3), 77.0, dtype=odt, device=DEV)
        qd = on_dev(q, pad).unflatten(1, (heads, dim)) if pad else q.to(DEV).view(rows, heads, dim)
        got = rts.indexer_logits(qd, on_dev(keys, pad), on_dev(w, 3), key_scales=ks.to(DEV) if use_ks else None,
                                 row_ends=ends.to(DEV) if use_ends else None, out=out)
        got = got.float().cpu()
        for t in range(rows):
            e = min(int(ends[t]), cols) if use_ends else cols
            want, bound = ref.logits(q[t].view(heads, dim), keys[:e], w[t], ks[:e] if use_ks else None)
            if odt == torch.bfloat16:
                bound = bound * (1 + ref.BF16) + want.abs() * ref.BF16
            ref.assert_close(got[t, :e], want, bound, f"row {t}")
            assert (got[t, e:] == 77.0).all(), "columns behind the row's end were written"


@pytest.mark.parametrize("heads", [32, 5, 33])
def test_indexer_logits_non_finite(rts, heads):
    say("logits: NaN and infinities stay in their column, and infinities are ordinary", heads)
    g = gen(3)
    q = torch.rand(4, heads, 128, generator=g).bfloat16() + 0.5   # positive: an infinity keeps its sign
    keys = torch.randn(200, 128, generator=g).bfloat16()
    w = torch.rand(4, heads, generator=g) + 0.5
    w[1] = -w[1]
    keys[17, 3] = math.nan
    keys[40, 0] = math.inf
    keys[41, 5] = -math.inf
    keys[199] = math.nan
    ends = torch.tensor([200, 199, 40, 17], dtype=torch.int32)
    got = rts.indexer_logits(q.to(DEV), keys.to(DEV), w.to(DEV), row_ends=ends.to(DEV)).cpu()
    fine = torch.ones(200, dtype=torch.bool)
    fine[[17, 40, 41, 199]] = False
    for t in range(4):
        e = int(ends[t])
        ok = fine[:e]
        want, bound = ref.logits(q[t], keys[:e][ok], w[t], None)
        ref.assert_close(got[t, :e][ok], want, bound, f"row {t}")
        at = torch.arange(e)
        assert torch.isnan(got[t, :e][(at == 17) | (at == 199)]).all()
        assert (got[t, :e][at == 40] == (-math.inf if t == 1 else math.inf)).all()
        assert (got[t, :e][at == 41] == 0).all()


def test_indexer_logits_e4m3_nan(rts):
    say("logits: e4m3 NaN stays in its column and its row")
    q, keys, w, ks = index_inputs(3, 3, 32, 128, 70, torch.float8_e4m3fn)
    keys.view(torch.uint8)[33, 100] = 0x7F
    q.view(torch.uint8)[2, 5] = 0xFF
    got = rts.indexer_logits(q.to(DEV).view(3, 32, 128), keys.to(DEV), w.contiguous().to(DEV),
                             key_scales=ks.to(DEV)).cpu()
    assert torch.isnan(got[:, 33]).all() and torch.isnan(got[2]).all()
    ok = torch.arange(70) != 33
    for t in range(2):
        want, bound = ref.logits(q[t].view(32, 128), keys[ok], w[t], ks[ok])
        ref.assert_close(got[t, ok], want, bound, f"row {t}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "e4m3"])
@pytest.mark.parametrize("counts,heads,dim,block,ctx", [([1], 64, 128, 64, 500), ([1] * 9, 32, 128, 16, 300),
                                                       ([3, 3, 3], 64, 64, 48, 400), ([5, 1, 0, 9], 24, 128, 1, 70),
                                                       ([2, 30], 128, 128, 128, 1000)])
def test_indexer_logits_paged(rts, dtype, counts, heads, dim, block, ctx):
    say("logits paged", dtype, counts, heads, dim, block, ctx)
    reqs, rows = len(counts), sum(counts) + 2  # two padding tokens
    rng = np.random.default_rng(rows)
    stride = block + 1
    cols_t = -(-(ctx + max(counts)) // block)
    cache_rows = reqs * cols_t * stride
    q, keys, w, ks = index_inputs(rows, rows, heads, dim, cache_rows, dtype)
    table = rng.permutation(reqs * cols_t).astype(np.int32).reshape(reqs, cols_t)
    lens = rng.integers(1, ctx + 1, size=reqs)
    lens[0] = ctx
    if cols_t > 2:
        table[0, 1] = -1                      # a missing page
        table[-1, 0] = reqs * cols_t + 50     # a page outside the cache
    req, ends = [], []
    for r, n in enumerate(counts):
        for j in range(n):
            req.append(r)
            ends.append(int(lens[r]) + j + 1)
    req += [-1, reqs]
    ends += [5, 5]
    width = max(ends)
    out = torch.full((rows, width), 77.0, device=DEV)
    rts.indexer_logits_paged(q.to(DEV).view(rows, heads, dim), keys.to(DEV), w.contiguous().to(DEV), i32(req),
                             i32(ends), torch.from_numpy(table).to(DEV), block, width, key_scales=ks.to(DEV),
                             stride_rows=stride, out=out)
    got = out.cpu()
    for t in range(rows):
        if not 0 <= req[t] < reqs:
            assert (got[t] == 77.0).all()
            continue
        where = [ref.phys(table[req[t]].tolist(), p, block, stride, cache_rows) for p in range(ends[t])]
        at = torch.tensor([0 if x is None else x for x in where])
        want, bound = ref.logits(q[t].view(heads, dim), keys[at], w[t], ks[at])
        want[torch.tensor([x is None for x in where])] = math.nan
        ref.assert_close(got[t, :ends[t]], want, bound, f"token {t}")
        assert (got[t, ends[t]:] == 77.0).all()


def test_indexer_logits_far_offsets(rts):
    say("logits: a key cache past 4 GiB, output rows past 4 GiB")
    rows = 40_000_000
    keys = torch.zeros(rows, 128, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    block = 64
    at = torch.tensor([rows // block - 1, 3, rows // block - 2, 0])
    q, some, w, _ = index_inputs(8, 2, 32, 128, 4 * block, torch.float8_e4m3fn)
    for i, b in enumerate(at.tolist()):
        keys.view(torch.uint8)[b * block:(b + 1) * block] = some[i * block:(i + 1) * block].view(torch.uint8).to(DEV)
    far = torch.empty(2, 1_300_000_000, device=DEV)[:, :256]
    got = rts.indexer_logits_paged(q.to(DEV).view(2, 32, 128), keys, w.contiguous().to(DEV), i32([0, 0]), i32([256, 255]),
                                   at.int().to(DEV)[None], block, 256, out=far).cpu()
    for t, e in ((0, 256), (1, 255)):
        want, bound = ref.logits(q[t].view(32, 128), some[:e], w[t], None)
        ref.assert_close(got[t, :e], want, bound, f"row {t}")


def test_paged_calls_without_pages(rts):
    say("paged calls on an empty table and an empty cache")
    q, keys, w, _ = index_inputs(4, 3, 32, 128, 64, torch.bfloat16)
    for keys_d, table in ((keys.to(DEV), torch.empty(2, 0, dtype=torch.int32, device=DEV)),
                          (keys[:0].to(DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV))):
        got = rts.indexer_logits_paged(q.to(DEV).view(3, 32, 128), keys_d, w.contiguous().to(DEV), i32([0, 1, 1]),
                                       i32([5, 40, 0]), table, 16, 40, out=torch.zeros(3, 40, device=DEV)).cpu()
        assert torch.isnan(got[0, :5]).all() and torch.isnan(got[1]).all()
        assert (got[0, 5:] == 0).all() and (got[2] == 0).all()
    lq, cache = latent_inputs(5, 3, 16, 512, 64)
    for cache_d, table in ((cache.to(DEV), torch.empty(2, 0, dtype=torch.int32, device=DEV)),
                           (cache[:0].to(DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV))):
        out, lse = rts.latent_attend_paged(lq.to(DEV), cache_d, i32([0, 1, 3]), i32([9, 20]), table, 16, 0.07)
        assert (out == 0).all() and (lse == -math.inf).all()


# ---------------------------------------------------------- latent attention

def latent_inputs(seed, rows, heads, latent, cache_rows, sharp=1.0):
    g = gen(seed)
    d = latent + 64
    q = (torch.randn(rows, heads, d, generator=g) * sharp).bfloat16()
    cache = torch.randn(cache_rows, d, generator=g).bfloat16()
    return q, cache


def padded3(t, row_pad, head_pad):
    """A GPU copy of [rows, heads, d] with padded head and row strides (multiples of 8)."""
    rows, heads, d = t.shape
    wide = torch.full((rows, heads * (d + head_pad) + row_pad), math.nan, dtype=t.dtype, device=DEV)
    view = wide[:, : heads * (d + head_pad)].unflatten(1, (heads, d + head_pad))[:, :, :d]
    view.copy_(t)
    return view


def check_rows(rts, q, cache, ids, counts, scale, latent, workspace="auto", qd=None, cd=None):
    rows, heads, _ = q.shape
    out, lse = rts.latent_attend_rows(q.to(DEV) if qd is None else qd, cache.to(DEV) if cd is None else cd,
                                      ids.to(DEV), scale, d_latent=latent,
                                      counts=None if counts is None else counts.to(DEV), workspace=workspace)
    out, lse = out.cpu(), lse.cpu()
    for t in range(rows):
        n = ids.shape[1] if counts is None else min(max(int(counts[t]), 0), ids.shape[1])
        at = ids[t, :n].long()
        at = at[(at >= 0) & (at < cache.shape[0])]
        o, l, ob, lb = ref.attend(q[t], cache[at], scale, latent)
        ref.assert_close(out[t], o, ob, f"out of row {t}")
        ref.assert_close(lse[t], l, lb, f"lse of row {t}")
    return out, lse


@pytest.mark.parametrize("latent", [512, 256])
@pytest.mark.parametrize("rows,heads,k", [(1, 1, 1), (1, 16, 33), (3, 16, 500), (2, 20, 64), (5, 32, 31), (3, 48, 97),
                                          (2, 64, 256), (4, 96, 40), (2, 128, 300), (1, 130, 70), (1, 128, 2048)])
def test_latent_rows(rts, latent, rows, heads, k):
    say("latent rows", latent, rows, heads, k)
    q, cache = latent_inputs(rows * k + heads, rows, heads, latent, 3000)
    ids = torch.randint(0, 3000, (rows, k), generator=gen(k)).int()
    check_rows(rts, q, cache, ids, None, 192 ** -0.5, latent)
    check_rows(rts, q, cache, ids, None, 192 ** -0.5, latent, workspace=None)


def test_latent_rows_counts_and_bad_ids(rts):
    say("latent rows: counts, -1 tails, ids outside the cache, NaN in rows that are not listed")
    q, cache = latent_inputs(11, 8, 40, 512, 600)
    k = 200
    ids = torch.randint(0, 500, (8, k), generator=gen(5)).int()
    cache[500:] = math.nan  # never listed within a row's count, but a neighbour in memory
    counts = torch.tensor([k, 0, 1, 33, -4, k + 9, 64, 100], dtype=torch.int32)
    ids[0, 3:7] = -1
    ids[0, 9] = 600
    ids[0, 10] = 2 ** 31 - 1
    ids[2, 1:] = 550        # behind the count: not read
    ids[3, 33:] = 550
    ids[6, :64] = -1        # a row of which nothing is left
    ids[7, :] = 5           # the same id over and over
    check_rows(rts, q, cache, ids, counts, 0.07, 512)
    check_rows(rts, q, cache, ids, counts, 0.07, 512, workspace=None)
    check_rows(rts, q, cache, ids[:, :0].contiguous(), None, 0.07, 512)   # no entries at all
    empty = torch.empty(0, 576, dtype=torch.bfloat16)
    check_rows(rts, q, empty, ids, None, 0.07, 512)                      # no cache


@pytest.mark.parametrize("sharp", [0.0, 30.0])
def test_latent_rows_flat_and_sharp_scores(rts, sharp):
    say("latent rows: scores all equal, and far apart in rising and falling order", sharp)
    q, cache = latent_inputs(12, 3, 32, 512, 700, sharp)
    ids = torch.arange(700).int().repeat(3, 1)
    z = cache.double() @ q[1, 0].double()
    ids[1] = z.argsort().int()
    ids[2] = (cache.double() @ q[2, 5].double()).argsort(descending=True).int()
    check_rows(rts, q, cache, ids, None, 0.07, 512)
    check_rows(rts, q, cache, ids, None, -0.07, 512)


def test_latent_rows_strides(rts):
    say("latent rows: strided q, cache and ids")
    q, cache = latent_inputs(13, 5, 24, 512, 300)
    wide = torch.full((300, 576 + 24), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, :576] = cache.to(DEV)
    ids = torch.randint(0, 300, (5, 90), generator=gen(1)).int()
    wide_ids = torch.full((5, 101), 2 ** 30, dtype=torch.int32)
    wide_ids[:, :90] = ids
    out, _ = check_rows(rts, q, cache, ids, None, 0.07, 512, qd=padded3(q, 16, 8), cd=wide[:, :576])
    by_head = q.permute(1, 0, 2).contiguous().to(DEV).permute(1, 0, 2)  # heads outermost in memory
    got, _ = rts.latent_attend_rows(by_head, wide[:, :576], wide_ids.to(DEV)[:, :90], 0.07)
    assert torch.equal(got.cpu(), out)


def test_latent_rows_infinite_weightless_rows(rts):
    say("latent rows: a listed NaN row reaches exactly the rows that list it")
    q, cache = latent_inputs(14, 4, 16, 512, 200)
    cache[7] = math.nan
    ids = torch.randint(8, 200, (4, 70), generator=gen(2)).int()
    ids[2, 50] = 7
    out, lse = rts.latent_attend_rows(q.to(DEV), cache.to(DEV), ids.to(DEV), 0.07)
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()
    keep = torch.tensor([0, 1, 3])
    check = check_rows(rts, q[keep], cache, ids[keep], None, 0.07, 512)
    assert torch.equal(check[0], out[keep].cpu())


def test_latent_rows_far_offsets(rts):
    say("latent rows: a cache past 4 GiB")
    cache_rows = 4_000_000
    cd = torch.zeros(cache_rows, 576, dtype=torch.bfloat16, device=DEV)
    at = torch.randperm(cache_rows, generator=gen(3))[:64]
    at[:2] = torch.tensor([0, cache_rows - 1])
    q, some = latent_inputs(15, 2, 16, 512, 64)
    cd[at.to(DEV)] = some.to(DEV)
    out, lse = rts.latent_attend_rows(q.to(DEV), cd, at.int().repeat(2, 1).to(DEV), 0.07)
    near = check_rows(rts, q, some, torch.arange(64).int().repeat(2, 1), None, 0.07, 512)
    assert torch.equal(out.cpu(), near[0]) and torch.equal(lse.cpu(), near[1])


def paged_setup(seed, ctx, new, heads, latent, block, stride=None, pad_tokens=0):
    rng = np.random.default_rng(seed)
    stride = block if stride is None else stride
    reqs = len(ctx)
    cols = max(1, max(-(-(c + n) // block) for c, n in zip(ctx, new)))
    table = rng.permutation(reqs * cols).astype(np.int32).reshape(reqs, cols)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q, cache = latent_inputs(seed, int(starts[-1]) + pad_tokens, heads, latent, reqs * cols * stride)
    return q, cache, starts, table, stride


def check_paged(rts, q, cache, starts, ctx, table, block, stride, scale, latent, tree=None, workspace="auto",
                max_len=None):
    tokens, heads, _ = q.shape
    out = torch.full((tokens, heads, latent), 55.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((tokens, heads), 55.0, device=DEV)
    td = None if tree is None else torch.tensor([x - (1 << 64) if x >> 63 else x for x in tree], dtype=torch.int64,
                                                device=DEV)
    rts.latent_attend_paged(q.to(DEV), cache.to(DEV), i32(starts.tolist()), i32(ctx), torch.from_numpy(table).to(DEV),
                            block, scale, d_latent=latent, stride_rows=stride, tree=td, max_len=max_len, out=out,
                            lse=lse, workspace=workspace)
    got, got_lse = out.cpu(), lse.cpu()
    for r in range(len(ctx)):
        for t in range(starts[r], starts[r + 1]):
            j, n = t - starts[r], starts[r + 1] - starts[r]
            c = max(ctx[r], 0)
            pos = list(range(c))
            if tree is None:
                pos += list(range(c, c + j + 1))
            else:
                pos += [c + b for b in range(min(n, 64)) if (tree[t] >> b) & 1]
            at = [ref.phys(table[r].tolist(), p, block, stride, cache.shape[0]) for p in pos]
            at = torch.tensor([x for x in at if x is not None], dtype=torch.int64)
            o, l, ob, lb = ref.attend(q[t], cache[at], scale, latent)
            ref.assert_close(got[t], o, ob, f"out of token {t} (request {r})")
            ref.assert_close(got_lse[t], l, lb, f"lse of token {t} (request {r})")
    end = int(starts[len(ctx)])
    assert (got[end:] == 55.0).all() and (got_lse[end:] == 55.0).all(), "rows behind the last token were written"
    return got, got_lse


@pytest.mark.parametrize("ctx,new,heads,latent,block,pad", [
    ([0], [1], 16, 512, 64, 0), ([1], [1], 1, 256, 1, 0), ([500, 3, 64, 0], [1, 1, 1, 1], 16, 512, 64, 3),
    ([31, 32, 33], [1, 2, 3], 32, 512, 16, 0), ([100, 0, 7, 250], [5, 0, 64, 1], 20, 512, 48, 2),
    ([700], [1], 128, 512, 64, 0), ([90, 200], [3, 2], 128, 256, 32, 1), ([40], [130], 8, 512, 16, 0),
    ([1000, 10], [2, 2], 64, 512, 128, 0), ([60, 61, 62], [1, 4, 1], 140, 512, 64, 0)])
def test_latent_paged(rts, ctx, new, heads, latent, block, pad):
    say("latent paged", ctx, new, heads, latent, block, pad)
    q, cache, starts, table, stride = paged_setup(sum(ctx) + heads, ctx, new, heads, latent, block, block + 2, pad)
    a = check_paged(rts, q, cache, starts, ctx, table, block, stride, 0.07, latent)
    check_paged(rts, q, cache, starts, ctx, table, block, stride, 0.07, latent, workspace=None)
    b = check_paged(rts, q, cache, starts, ctx, table, block, stride, 0.07, latent,
                    max_len=max(c + n for c, n in zip(ctx, new)))
    del a, b


def test_latent_paged_many_and_very_ragged_requests(rts):
    say("latent paged: 200 requests, some without tokens; one long request among short ones")
    rng = np.random.default_rng(3)
    ctx = rng.integers(0, 90, size=200).tolist()
    new = rng.integers(0, 3, size=200).tolist()
    q, cache, starts, table, stride = paged_setup(17, ctx, new, 16, 256, 16)
    check_paged(rts, q, cache, starts, ctx, table, 16, stride, 0.07, 256)
    check_paged(rts, q, cache, starts, ctx, table, 16, stride, 0.07, 256, workspace=None)
    ctx, new = [5000, 0, 3, 40, 700, 1], [1, 1, 0, 2, 1, 1]
    q, cache, starts, table, stride = paged_setup(18, ctx, new, 40, 512, 64)
    for max_len in (5001, 64, 0, 1 << 40):  # any bound gives right results
        check_paged(rts, q, cache, starts, ctx, table, 64, stride, 0.07, 512, max_len=max_len)


def test_latent_many_heads(rts):
    say("latent: 1024 heads")
    q, cache = latent_inputs(19, 1, 1024, 256, 50)
    check_rows(rts, q, cache, torch.arange(50).int()[None], None, 0.07, 256)


def test_latent_calls_at_once(rts):
    say("latent: calls on two streams at once, each with its own workspace")
    q, cache = latent_inputs(20, 4, 32, 512, 3000)
    qd, cd = q.to(DEV), cache.to(DEV)
    lists = [torch.randint(0, 3000, (4, 1500), generator=gen(k)).int().to(DEV) for k in range(2)]
    want = [rts.latent_attend_rows(qd, cd, ids, 0.07) for ids in lists]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k in range(2):
            got[k].append(rts.latent_attend_rows(qd, cd, lists[k], 0.07, stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for o, l in got[k]:
            assert torch.equal(o, want[k][0]) and torch.equal(l, want[k][1])


@pytest.mark.parametrize("ctx,new,heads,block", [([200, 0, 77], [8, 3, 1], 16, 16), ([129], [64], 4, 64),
                                                 ([30, 400], [70, 5], 2, 32), ([0, 0], [6, 6], 128, 64)])
def test_latent_tree(rts, ctx, new, heads, block):
    say("latent tree", ctx, new, heads, block)
    q, cache, starts, table, stride = paged_setup(sum(new) + heads, ctx, new, heads, 512, block)
    rng = np.random.default_rng(7)
    tree = []
    for n in new:
        mine = []
        for j in range(n):
            up = mine[rng.integers(0, j)] if j else 0
            mine.append(up | (1 << j if j < 64 else 0))
        tree += mine
    tree[0] = 0                      # sees the cached tokens only (none at all where there are none)
    tree[-1] = (1 << 64) - 1         # drafts behind itself too, and bits past the request's drafts
    check_paged(rts, q, cache, starts, ctx, table, block, stride, 0.07, 512, tree=tree)
    check_paged(rts, q, cache, starts, ctx, table, block, stride, 0.07, 512, tree=tree, workspace=None)


def test_latent_paged_missing_pages(rts):
    say("latent paged: missing pages, a table that ends early, negative lengths")
    ctx, new, block = [300, 90, -5], [2, 3, 4], 16
    q, cache, starts, table, stride = paged_setup(5, [300, 90, 0], new, 16, 512, block)
    table[0, 2] = -1
    table[0, 7] = 10 ** 6
    table[1, :] = -1
    check_paged(rts, q, cache, starts, ctx, table, block, stride, 0.07, 512)
    check_paged(rts, q, cache, starts, ctx, np.ascontiguousarray(table[:, :5]), block, stride, 0.07, 512)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_latent_paged_masked_values_do_not_reach_results(rts, bad):
    say("latent paged: non-finite vectors in masked places", bad)
    ctx, new, block = [70, 0, 33], [6, 5, 40], 16
    q, cache, starts, table, stride = paged_setup(6, ctx, new, 16, 512, block)
    clean = cache.clone()
    tree = []
    for r, n in enumerate(new):
        tree += [1 << j for j in range(n)]
        # the last draft's vector, and everything in the cache behind the request
        for p in range(ctx[r] + n - 1, table.shape[1] * block):
            cache[ref.phys(table[r].tolist(), p, block, stride, cache.shape[0])] = bad
    for mask in (None, tree):
        td = None if mask is None else torch.tensor(mask, dtype=torch.int64, device=DEV)
        res = []
        for c in (cache, clean):
            res.append(rts.latent_attend_paged(q.to(DEV), c.to(DEV), i32(starts.tolist()), i32(ctx),
                                               torch.from_numpy(table).to(DEV), block, 0.07, tree=td))
        seen = torch.zeros(q.shape[0], dtype=torch.bool)
        seen[starts[1:] - 1] = True  # only a request's last token sees its own vector
        for x, y in zip(res[0], res[1]):
            assert torch.equal(x.cpu()[~seen], y.cpu()[~seen])


def test_latent_streams_and_replay(rts):
    say("latent: other streams, two captured graphs, replays after new lengths")
    ctx, new, block = [300, 40], [1, 1], 16
    q, cache, starts, table, stride = paged_setup(8, ctx, new, 16, 512, block)
    qd, cd, sd, td = q.to(DEV), cache.to(DEV), i32(starts.tolist()), torch.from_numpy(table).to(DEV)
    cx = i32(ctx)
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=DEV)
    ids = torch.randint(0, cache.shape[0], (2, 600), generator=gen(4)).int().to(DEV)

    def paged(o):
        return rts.latent_attend_paged(qd, cd, sd, cx, td, block, 0.07, out=o)

    def rows():
        return rts.latent_attend_rows(qd, cd, ids, 0.07)

    paged(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = rts.latent_attend_rows(qd, cd, ids, 0.07, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(on_side, rows()))
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        paged(out)
    with torch.cuda.graph(gb):
        rows_out = rows()
    want_rows = rows()
    for c in ([300, 40], [1, 200], [0, 0], [299, 5]):
        cx.copy_(i32(c))
        ga.replay()
        gb.replay()
        fresh = torch.empty_like(out)
        paged(fresh)
        torch.cuda.synchronize()
        assert torch.equal(out, fresh)
        assert all(torch.equal(x, y) for x, y in zip(rows_out, want_rows))


# --------------------------------------------------------------- rank merge

@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                             (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("world,rows,heads,dim", [(1, 1, 1, 8), (2, 3, 16, 512), (4, 5, 7, 256), (8, 2, 128, 512),
                                                  (64, 3, 3, 24), (3, 1, 1, 2048)])
def test_merge_attend(rts, dtype, out_dtype, world, rows, heads, dim):
    say("merge", dtype, out_dtype, world, rows, heads, dim)
    g = gen(world + dim)
    parts = torch.randn(world, rows, heads, dim, generator=g).to(dtype)
    lse = torch.randn(world, rows, heads, generator=g) * 4
    lse[torch.rand(lse.shape, generator=g) < 0.2] = -math.inf
    lse[:, 0, 0] = -math.inf
    pd = parts.clone()
    pd[torch.isinf(lse)] = math.nan  # a rank without rows may leave anything there
    out, total = rts.merge_attend_rank_major(pd.to(DEV), lse.to(DEV), out_dtype=out_dtype)
    o, l, ob, lb = ref.merge(parts, lse)
    if out_dtype == torch.bfloat16:
        ob = ob * (1 + ref.BF16) + o.abs() * ref.BF16
    ref.assert_close(out, o, ob, "out")
    ref.assert_close(total, l, lb, "lse")


def test_merge_attend_nan(rts):
    say("merge: a NaN part beside empty ones stays NaN")
    parts = torch.randn(3, 2, 4, 64, generator=gen(9))
    lse = torch.full((3, 2, 4), -math.inf)
    lse[1, 0] = math.nan
    lse[2, 1] = 3.0
    out, total = rts.merge_attend_rank_major(parts.to(DEV), lse.to(DEV))
    assert torch.isnan(out[0]).all() and torch.isnan(total[0]).all()
    assert torch.equal(out[1].cpu(), parts[2, 1]) and (total[1] == 3.0).all()


# ------------------------------------------------------------- all together

def test_step_of_sparse_attention(rts):
    """One step as a serving loop runs it: slots, cache writes, logits, select, rows, attention; then
    the same attention from two ranks that own every other token."""
    import oracle
    say("a step: slots -> logits -> select -> rows -> attention -> merge of two ranks")
    g = gen(21)
    ctx, new, block, heads, k = [600, 35, 0, 257], [1, 3, 20, 1], 16, 16, 64
    reqs, tokens, cols_t = 4, 28, 48
    have = [-(-c // block) for c in ctx]
    ids = torch.randperm(reqs * cols_t, generator=g).int()
    table = torch.full((reqs, cols_t), -1, dtype=torch.int32)
    at = 0
    for r in range(reqs):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    td, free = table.to(DEV), ids[at:].contiguous().to(DEV)
    cache_rows = reqs * cols_t * block
    latent = torch.randn(cache_rows, 576, generator=g).bfloat16().to(DEV)
    keys = torch.randn(cache_rows, 128, generator=g).to(torch.float8_e4m3fn).to(DEV)
    scales = (torch.rand(cache_rows, generator=g) + 0.5).to(DEV)
    m = rts.assign_slots(i32(ctx), i32(new), tokens, td, free, block)
    live = m.slots >= 0
    latent[m.slots[live].long()] = torch.randn(25, 576, generator=g).bfloat16().to(DEV)
    keys.view(torch.uint8)[m.slots[live].long()] = (
        torch.randn(25, 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV))
    q_index = torch.randn(tokens, 32, 128, generator=g).to(torch.float8_e4m3fn).to(DEV)
    w = torch.randn(tokens, 32, generator=g).to(DEV)
    q = torch.randn(tokens, heads, 576, generator=g).bfloat16().to(DEV)
    width = max(ctx) + max(new)
    logits = rts.indexer_logits_paged(q_index, keys, w, m.req_id, m.row_ends, td, block, width, key_scales=scales)
    picked = rts.topk_rows(logits, k, row_ends=m.row_ends)
    rows, valid = rts.emit_rows(picked, 1, 0, m.req_id, td, block, block)
    out, lse = rts.latent_attend_rows(q, latent, rows, 0.07, counts=valid)

    ends, req, tab = host(m.row_ends), host(m.req_id), host(td)
    exp_ids = oracle.topk_rows(host(logits), ends, k)
    assert_ids_equal(host(picked), exp_ids, "picked")
    lat, kc, sc = latent.cpu(), keys.cpu(), scales.cpu()
    for t in range(tokens):
        if req[t] < 0:
            assert (out[t] == 0).all() and (lse[t] == -math.inf).all() and (picked[t] == -1).all()
            continue
        where = torch.tensor([ref.phys(tab[req[t]].tolist(), p, block, block, cache_rows) for p in range(ends[t])])
        x, b = ref.logits(q_index[t].cpu(), kc[where], w[t].cpu(), sc[where])
        ref.assert_close(logits[t, :ends[t]], x, b, f"logits of token {t}")
        chosen = where[torch.from_numpy(exp_ids[t][exp_ids[t] >= 0]).long()]
        o, l, ob, lb = ref.attend(q[t].cpu(), lat[chosen], 0.07, 512)
        ref.assert_close(out[t], o, ob, f"out of token {t}")
        ref.assert_close(lse[t], l, lb, f"lse of token {t}")
        if ends[t] <= k:  # nothing was left out: the dense form sees the same rows
            assert len(chosen) == ends[t]
    dense, dense_lse = rts.latent_attend_paged(q, latent, m.query_starts, i32(ctx), td, block, 0.07)
    short = torch.from_numpy((ends <= k) & (req >= 0)).to(DEV)
    ref.assert_close(dense[short], out[short], 2 * ref.BF16 * (out[short].double().abs() + 1), "dense")
    ref.assert_close(dense_lse[short], lse[short], 1e-4 + 0 * lse[short].double(), "dense lse")

    # Two ranks: rank r holds the tokens with position % 2 == r at local index
    # position // 2, in a cache and a table of its own.
    parts, sums = [], []
    for r in range(2):
        local = torch.zeros(reqs * cols_t * block, 576, dtype=torch.bfloat16, device=DEV)
        tab_r = torch.arange(reqs * cols_t, dtype=torch.int32, device=DEV).view(reqs, cols_t)
        for i in range(reqs):
            n = ctx[i] + new[i]
            pos = torch.arange(r, n, 2)
            src = torch.tensor([ref.phys(tab[i].tolist(), int(p), block, block, cache_rows) for p in pos],
                               dtype=torch.int64)
            dst = i * cols_t * block + torch.arange(len(pos))
            local[dst.to(DEV)] = latent[src.to(DEV)]
        rr, vv = rts.emit_rows(picked, 2, r, m.req_id, tab_r, block, block)
        o, l = rts.latent_attend_rows(q, local, rr, 0.07, counts=vv)
        parts.append(o)
        sums.append(l)
    both, both_lse = rts.merge_attend_rank_major(torch.stack(parts), torch.stack(sums))
    for t in range(tokens):
        if req[t] < 0:
            assert (both[t] == 0).all()
            continue
        where = torch.tensor([ref.phys(tab[req[t]].tolist(), p, block, block, cache_rows) for p in range(ends[t])])
        chosen = where[torch.from_numpy(exp_ids[t][exp_ids[t] >= 0]).long()]
        o, l, ob, lb = ref.attend(q[t].cpu(), lat[chosen], 0.07, 512)
        # Each rank's result is rounded to bf16 once before the merge: half a
        # step of a part, at most the largest value of its rows.
        more = ref.BF16 * lat[chosen][:, :512].double().abs().amax(0)
        ref.assert_close(both[t], o, 2 * ob + more[None], f"merged out of token {t}")
        ref.assert_close(both_lse[t], l, 4 * lb + 1e-5, f"merged lse of token {t}")


def test_captured_step(rts):
    """The whole step in one graph, replayed after new lengths, queries and tables, with eager work
    between the replays."""
    say("a captured step, replayed")
    block, reqs, tokens, cols_t, k, width = 16, 3, 8, 20, 32, 300
    g = gen(31)
    cache_rows = reqs * cols_t * block
    latent = torch.randn(cache_rows, 576, generator=g).bfloat16().to(DEV)
    keys = torch.randn(cache_rows, 128, generator=g).bfloat16().to(DEV)
    q_index = torch.zeros(tokens, 16, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(tokens, 16, device=DEV)
    q = torch.zeros(tokens, 16, 576, dtype=torch.bfloat16, device=DEV)
    ctx, new = i32([0] * reqs), i32([0] * reqs)
    table = torch.zeros(reqs, cols_t, dtype=torch.int32, device=DEV)
    free = torch.arange(reqs * cols_t, dtype=torch.int32, device=DEV)

    def step():
        m = rts.assign_slots(ctx, new, tokens, table, free, block)
        logits = rts.indexer_logits_paged(q_index, keys, w, m.req_id, m.row_ends, table, block, width)
        picked = rts.topk_rows(logits, k, row_ends=m.row_ends)
        rows, valid = rts.emit_rows(picked, 1, 0, m.req_id, table, block, block)
        out, lse = rts.latent_attend_rows(q, latent, rows, 0.07, counts=valid)
        dense = torch.zeros_like(out)
        rts.latent_attend_paged(q, latent, m.query_starts, ctx, table, block, 0.07, out=dense)
        both = rts.merge_attend_rank_major(torch.stack([out, dense]), torch.stack([lse, lse]))
        return [*m, picked, out, lse, dense, *both]

    def set_inputs(seed):
        h = gen(seed)
        q_index.copy_(torch.randn(q_index.shape, generator=h))
        w.copy_(torch.randn(w.shape, generator=h))
        q.copy_(torch.randn(q.shape, generator=h))
        ctx.copy_(torch.randint(0, 290, (reqs,), generator=h))
        new.copy_(torch.randint(0, 4, (reqs,), generator=h))
        table.copy_(torch.randperm(reqs * cols_t, generator=h).view(reqs, cols_t))

    set_inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(1, 6):
        set_inputs(seed)
        before = table.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        table.copy_(before)
        for i, (x, y) in enumerate(zip(got, step())):
            assert torch.equal(x, y), (seed, i)
