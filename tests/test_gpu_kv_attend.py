"""kv_attend_paged against its definition in 64 bits."""

import math

import pytest

import beam_reference as ref
from gpu_common import say
from serving_reference import assert_close

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rand(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def check(rts, q, k, v, req, ends, table, block, scale, stride=None, window=0, ks=None, vs=None, max_len=None,
          workspace="auto", kd=None, vd=None, qd=None):
    """q, k, v on the CPU; kd, vd, qd: the tensors to hand over, where they differ.  Calls that may be split are made
    with a bound on the lengths too that has them split."""
    stride = block if stride is None else stride
    kd, vd = (k.to(DEV) if kd is None else kd), (v.to(DEV) if vd is None else vd)
    qd = q.to(DEV) if qd is None else qd
    def call(max_len):
        return rts.kv_attend_paged(
            qd, kd, vd, i32(req), i32(ends), i32(table) if table and table[0] else torch.empty(
                len(table), 0, dtype=torch.int32, device=DEV), block, scale, k_scales=None if ks is None else ks.to(DEV),
            v_scales=None if vs is None else vs.to(DEV), window=window, stride_rows=stride, max_len=max_len,
            workspace=workspace)

    got, lse = call(max_len)
    calls = [(got, lse)] + ([call(1 << 20)] if max_len is None and workspace == "auto" else [])
    torch.cuda.synchronize()
    rows, heads, dim = q.shape
    kv_heads = k.shape[1]
    group = heads // kv_heads
    want = [[], [], [], []]
    for t in range(rows):
        at = []
        if 0 <= req[t] < len(table):
            at = ref.seen_rows(table[req[t]], ends[t] - window if window else 0, ends[t], block, stride, k.shape[0])
        for h in range(kv_heads):
            s = scale * (1.0 if ks is None else float(ks[h]))
            f = 1.0 if vs is None else float(vs[h])
            o, l, ob, lb = ref.kv_attend(q[t, h * group:(h + 1) * group], k[at, h].float(), v[at, h].float(), s)
            for x, y in zip(want, (o * f, l, ob * abs(f), lb)):
                x.append(y)
    o, ob = (torch.stack(want[i]).view(rows, heads, dim) for i in (0, 2))
    l, lb = (torch.stack(want[i]).view(rows, heads) for i in (1, 3))
    for got, lse in reversed(calls):
        assert_close(got, o, ob, "out")
        assert_close(lse, l, lb, "lse")
    return got, lse


def setup(seed, ctx, heads, kv, dim, block, stride=None, dtype=torch.bfloat16, spare=0, each=1):
    g = torch.Generator().manual_seed(seed)
    stride = block if stride is None else stride
    cols = max(1, -(-max(ctx) // block)) + spare
    n = len(ctx) * cols
    table = torch.randperm(n, generator=g).view(len(ctx), cols).tolist()
    k, v = (rand(g, n * stride, kv, dim, dtype=dtype) for _ in range(2))
    q = rand(g, len(ctx) * each, heads, dim)
    req = [i for i in range(len(ctx)) for _ in range(each)]
    ends = [max(0, c - each + 1 + j) for c in ctx for j in range(each)]
    return q, k, v, req, ends, table


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ctx,heads,kv,block,stride", [
    ([1], 1, 1, 16, 16), ([33, 0, 64, 65], 8, 8, 16, 20), ([100, 31, 7], 12, 3, 24, 24), ([500], 32, 2, 1, 1),
    ([130, 1030], 40, 2, 64, 64), ([3000], 4, 1, 128, 128)])
def test_kv_attend(rts, dtype, dim, ctx, heads, kv, block, stride):
    say("kv", dtype, dim, ctx, heads, kv, block, stride)
    a = setup(dim + heads, ctx, heads, kv, dim, block, stride, dtype)
    ks = vs = None
    if dtype == E4M3:
        g = torch.Generator().manual_seed(1)
        ks, vs = torch.rand(kv, generator=g) + 0.5, torch.rand(kv, generator=g) - 0.5
    for ws in ("auto", None):
        check(rts, *a, block, dim ** -0.5, stride=stride, ks=ks, vs=vs, workspace=ws)


@pytest.mark.parametrize("window", [1, 31, 100, 840, 1300, 5000])
@pytest.mark.parametrize("each", [1, 3])
def test_window(rts, window, each):
    say("window", window, each)
    a = setup(window, [1, 400, 90, 1500], 16, 2, 128, 16, each=each)
    for ws in ("auto", None):
        check(rts, *a, 16, 0.09, window=window, workspace=ws)


def plan(rts, rows, heads, kv, dim, max_len, window=0):
    import ctypes
    p = (ctypes.c_int64 * 2)()
    i64 = ctypes.c_int64
    assert rts.raw_library().kv_attend_paged_plan(i64(rows), heads, kv, dim, 1, i64(max_len), i64(window), 1, p) == 0
    return p[0], p[1]


def test_pieces(rts):
    """Lengths at the borders of the pieces, and bounds on the lengths that are too low or too high."""
    target, least = plan(rts, 6, 8, 1, 64, 4096)
    assert target * least > 5000  # so all rows together are cut into the least pieces
    ctx = [4096] * 3
    a = list(setup(7, ctx, 8, 1, 64, 32))
    a[0] = a[0].repeat(2, 1, 1)
    a[3] = [0, 1, 2, 0, 1, 2]
    a[4] = [least, least + 1, 2 * least - 1, 4096, least - 1, 1]
    for max_len in (None, 0, 1, least, 5000, 1 << 40):
        check(rts, *a, 32, 0.125, max_len=max_len)


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 130, 700])
def test_pieces_of_many_and_very_ragged_rows(rts, rows):
    """One long row among short and empty ones, at every place where the sums over the rows go on."""
    g = torch.Generator().manual_seed(rows)
    q, k, v, _, _, table = setup(12, [3000, 40], 2, 1, 64, 16)
    q = rand(g, rows, 2, 64)
    for at in {0, rows // 2, rows - 1}:
        req, ends = [1] * rows, torch.randint(0, 41, (rows,), generator=g).tolist()
        req[at], ends[at] = 0, 3000
        check(rts, q, k, v, req, ends, table, 16, 0.125)


def test_longer_pieces(rts):
    """So many keys that the pieces are longer than the least."""
    target, least = plan(rts, 40, 8, 8, 64, 1 << 20)
    ctx = [3000 + 7 * i for i in range(40)]
    assert sum(ctx) > 2 * target * least
    check(rts, *setup(13, ctx, 8, 8, 64, 64), 64, 0.125)


def test_padded_batch_and_bad_requests(rts):
    q, k, v, req, ends, table = setup(3, [50, 20, 90, 10, 5, 40], 8, 2, 128, 16)
    req = [0, -1, 2, 6, 2 ** 31 - 1, 5]
    ends = [50, 20, -7, 10, 5, 2 ** 31 - 1]  # the last is cut at the table's end
    got, lse = check(rts, q, k, v, req, ends, table, 16, 0.1)
    for t in (1, 2, 3, 4):
        assert (got[t] == 0).all() and (lse[t] == -math.inf).all()
    # no table at all, no rows of a cache
    check(rts, q, k, v, req, ends, [[]] * 6, 16, 0.1)
    none = k[:0]
    check(rts, q, none, none, req, ends, table, 16, 0.1)
    out, _ = rts.kv_attend_paged(q[:0].to(DEV), k.to(DEV), v.to(DEV), i32([]), i32([]), i32(table), 16, 0.1)
    assert out.shape == (0, 8, 128)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_missing_pages_and_masked_values(rts, bad):
    """What is not seen never reaches a result: behind the end, before the window, pages without a block."""
    say("masked", bad)
    q, k, v, req, ends, table = setup(5, [75, 300], 8, 2, 128, 16, spare=2)
    table[1][3] = -1
    table[1][7] = 10 ** 6
    table[0][1] = 2 ** 31 - 1
    used = set()
    for r, e in zip(req, ends):
        used |= set(ref.seen_rows(table[r], e - 200, e, 16, 16, k.shape[0]))
    for r in range(k.shape[0]):
        if r not in used:
            k[r], v[r] = bad, bad
    for ws in ("auto", None):
        got, _ = check(rts, q, k, v, req, ends, table, 16, 0.1, window=200, workspace=ws)
        assert bool(torch.isfinite(got).all())


def test_infinities_that_are_seen(rts):
    """A score of -inf has no weight (and 0 times an infinity is NaN); NaN and +inf scores make the head NaN."""
    for ws in ("auto", None):
        q, k, v, req, ends, table = setup(6, [200, 40], 2, 2, 64, 16)
        q = q.abs()
        at = ref.seen_rows(table[0], 0, 200, 16, 16, k.shape[0])
        k[at[5], 0, 3] = -math.inf
        v[at[5], 0, 7] = math.inf
        k[at[100], 1, 9] = math.nan
        other = ref.seen_rows(table[1], 0, 40, 16, 16, k.shape[0])
        k[other[1], 0, 0] = math.inf
        k[other, 1, 0] = -math.inf  # every score of this head
        got, lse = rts.kv_attend_paged(q.to(DEV), k.to(DEV), v.to(DEV), i32(req), i32(ends), i32(table), 16, 0.1,
                                       workspace=ws)
        got, lse = got.cpu(), lse.cpu()
        nan = torch.isnan(got)
        assert nan[0, 0].tolist() == [i == 7 for i in range(64)] and math.isfinite(float(lse[0, 0]))
        assert bool(nan[0, 1].all()) and bool(torch.isnan(lse[0, 1]))
        assert bool(nan[1, 0].all())
        assert (got[1, 1] == 0).all() and float(lse[1, 1]) == -math.inf


@pytest.mark.parametrize("scale", [0.0, -0.2, 30.0, -2.0 ** 60, 2.0 ** -130])
def test_scales(rts, scale):
    say("scale", scale)
    a = setup(8, [90, 700], 6, 2, 64, 16)
    if abs(scale) < 1e6:
        for ws in ("auto", None):
            check(rts, *a, 16, scale, workspace=ws)
        return
    got, lse = rts.kv_attend_paged(a[0].to(DEV), a[1].to(DEV), a[2].to(DEV), i32(a[3]), i32(a[4]), i32(a[5]), 16, scale)
    for t in range(2):  # the one key of the greatest score, as far as 32-bit products tell
        at = ref.seen_rows(a[5][a[3][t]], 0, a[4][t], 16, 16, a[1].shape[0])
        for h in range(6):
            z = -(a[1][at, h // 3].double() @ a[0][t, h].double())
            best, next_best = z.topk(2).values.tolist()
            if best - next_best > 64 * ref.U * float(z.abs().max()):
                assert torch.equal(got[t, h].cpu(), a[2][at[int(z.argmax())], h // 3])
                assert abs(float(lse[t, h]) / -scale - best) <= 66 * ref.U * 64 * 4


def test_strides_and_layouts(rts):
    """Heads before positions in a block, keys beside values in one row, queries out of a wider product."""
    g = torch.Generator().manual_seed(2)
    ctx, heads, kv, dim, block = [70, 130], 8, 4, 64, 16
    q, k, v, req, ends, table = setup(9, ctx, heads, kv, dim, block)
    n = k.shape[0] // block
    for pair in (0, 1):
        if pair == 0:
            both = torch.empty(k.shape[0], 2, kv, dim, dtype=torch.bfloat16, device=DEV)
            kd, vd = both[:, 0], both[:, 1]
            kd.copy_(k)
            vd.copy_(v)
            stride = block
        else:  # [blocks, kv, block, dim]: rows of dim elements, a head's are block * dim further on
            pages = [torch.empty(n, kv, block, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            for p, x in zip(pages, (k, v)):
                p.copy_(x.view(n, block, kv, dim).transpose(1, 2))
            rows = (n - 1) * kv * block + block
            kd, vd = (p.as_strided((rows, kv, dim), (dim, block * dim, 1)) for p in pages)
            stride = kv * block
        wide = torch.zeros(2, heads * dim + 128 + 64, dtype=torch.bfloat16, device=DEV)
        qd = wide[:, 64:64 + heads * dim].view(2, heads, dim)
        qd.copy_(q)
        out, lse = rts.kv_attend_paged(qd, kd, vd, i32(req), i32(ends), i32(table), block, 0.1, stride_rows=stride)
        want, want_lse = check(rts, q, k, v, req, ends, table, block, 0.1)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_many_rows(rts):
    """More rows than the chip has places for, all of the same short request."""
    q, k, v, _, _, table = setup(10, [37], 2, 1, 64, 16)
    rows = 3000
    q = rand(torch.Generator().manual_seed(1), rows, 2, 64)
    ends = [t % 38 for t in range(rows)]
    check(rts, q, k, v, [0] * rows, ends, table, 16, 0.125)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_far_offsets(rts, dtype):
    """Rows past 2^32 bytes of a cache, and a block stride that passes 32 bits with a large block id."""
    kv, dim = 8, 128
    rows = 5_000_000 if dtype == E4M3 else 2_500_000
    k = torch.zeros(rows, kv, dim, dtype=dtype, device=DEV)
    v = torch.zeros(rows, kv, dim, dtype=dtype, device=DEV)
    g = torch.Generator().manual_seed(4)
    ks, vs = rand(g, 48, kv, dim, dtype=dtype), rand(g, 48, kv, dim, dtype=dtype)
    last = rows // 16 - 1
    for i, b in enumerate((last, 0, last - 7)):
        k[b * 16:b * 16 + 16] = ks[i * 16:i * 16 + 16].to(DEV)
        v[b * 16:b * 16 + 16] = vs[i * 16:i * 16 + 16].to(DEV)
    q = rand(g, 1, 16, dim)
    got, lse = rts.kv_attend_paged(q.to(DEV), k, v, i32([0]), i32([45]), i32([[last, 0, last - 7]]), 16, 0.1)
    want, want_lse = check(rts, q, ks, vs, [0], [45], [[0, 1, 2]], 16, 0.1)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    got, lse = rts.kv_attend_paged(q.to(DEV), k, v, i32([0]), i32([40]), i32([[2 ** 31 - 1, 0, 3]]), 16, 0.1,
                                   stride_rows=2 ** 40)
    want, want_lse = check(rts, q, ks[16:32], vs[16:32], [0], [16], [[0]], 16, 0.1)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


def test_streams_replay_and_calls_at_once(rts):
    q, k, v, req, ends, table = setup(11, [700, 40, 0, 1300], 8, 2, 128, 16)
    qd, kd, vd, r, e, t = q.to(DEV), k.to(DEV), v.to(DEV), i32(req), i32(ends), i32(table)
    call = lambda **kw: rts.kv_attend_paged(qd, kd, vd, r, e, t, 16, 0.1, **kw)  # noqa: E731
    want, want_lse = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams * 3:
        s.wait_stream(torch.cuda.current_stream())
        got.append(call(stream=s))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    n = rts.kv_attend_paged_workspace_size(torch.bfloat16, 4, 8, 2, 128, 1300)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(qd), torch.empty(4, 8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, lse=lse, workspace=ws, max_len=1300)
    for lens in ([700, 40, 0, 1300], [0, 5, 33, 128], [1, 1, 1, 1299]):
        e.copy_(torch.tensor(lens))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        eager, eager_lse = call(max_len=1300)
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse)
        check(rts, q, k, v, req, lens, table, 16, 0.1)


@pytest.mark.parametrize("heads,kv", [(128, 1), (34, 2), (3, 3)])
def test_groups_of_heads(rts, heads, kv):
    """Many query heads a key head, and numbers that leave a block of 16 partly empty."""
    for ws in ("auto", None):
        check(rts, *setup(heads, [150, 33, 2], heads, kv, 64, 16), 16, 0.125, workspace=ws)


def test_more_rows_than_are_split(rts):
    q, k, v, _, _, table = setup(14, [200], 1, 1, 64, 16)
    rows = 4100
    assert plan(rts, rows, 1, 1, 64, 1 << 20)[0] == 0 and plan(rts, 4096, 1, 1, 64, 1 << 20)[0] > 0
    q = rand(torch.Generator().manual_seed(2), rows, 1, 64)
    ends = [(7 * t) % 201 for t in range(rows)]
    check(rts, q, k, v, [0] * rows, ends, table, 16, 0.125)


def test_key_scales_of_any_sign(rts):
    q, k, v, req, ends, table = setup(15, [60, 300], 8, 4, 64, 16, dtype=E4M3)
    ks, vs = torch.tensor([-0.7, 0.0, 1e-3, 2.0]), torch.tensor([0.0, -1.5, 300.0, 1e-6])
    for scale in (0.2, -0.2):
        check(rts, q, k, v, req, ends, table, 16, scale, ks=ks, vs=vs)


def test_longest_contexts(rts):
    """Positions up to 2^31 - 1, few of which have a row: blocks of 2^30 tokens over a small cache."""
    g = torch.Generator().manual_seed(16)
    k, v, q = rand(g, 100, 1, 64), rand(g, 100, 1, 64), rand(g, 2, 2, 64)
    end = 2 ** 31 - 1
    for window in (0, 2 ** 30 + 40):
        got, lse = rts.kv_attend_paged(q.to(DEV), k.to(DEV), v.to(DEV), i32([0, 0]), i32([end, 2 ** 30 + 7]), i32([[0, 0]]),
                                       2 ** 30, 0.125, window=window)
        for t, e in ((0, end), (1, 2 ** 30 + 7)):
            seen = [p % 2 ** 30 for p in [*range(100), *range(2 ** 30, 2 ** 30 + 100)]
                    if p < e and (not window or p >= e - window)]
            o, l, ob, lb = ref.kv_attend(q[t], k[seen, 0], v[seen, 0], 0.125)
            assert_close(got[t], o, ob, f"out {window} {t}")
            assert_close(lse[t], l, lb, f"lse {window} {t}")
