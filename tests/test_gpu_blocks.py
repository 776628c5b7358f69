"""fork_blocks, compact_blocks and copy_blocks against their definitions on lists."""

import pytest

import beam_reference as ref
from gpu_common import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def padded(table, pad):
    wide = torch.full((len(table), len(table[0]) + pad), 123456789, dtype=torch.int32, device=DEV)
    t = wide[:, :len(table[0])]
    t.copy_(torch.tensor(table, dtype=torch.int32))
    return t


def assert_same(got, want, what):
    for name, w in want.items():
        g = getattr(got, name).tolist()
        assert g == w, f"{what}: {name} differs, first at " + str(
            next((i, a, b) for i, (a, b) in enumerate(zip(g, w)) if a != b) if len(g) == len(w) else (len(g), len(w)))


def setup(seed, reqs, beams, max_ctx, block, pool, held, cols=None):
    """Tables whose beams share a prompt, with ids all over the pool and beyond it, and unused entries of any value."""
    g = torch.Generator().manual_seed(seed)
    cols = cols or -(-max_ctx // block) + 1
    order = torch.randperm(pool, generator=g).tolist()
    take = iter(order * 50)
    table, ctx = [], []
    for _ in range(reqs):
        c = int(torch.randint(0, max_ctx + 1, (1,), generator=g))
        shared = [next(take) for _ in range(c // block // 2)]
        for _ in range(beams):
            row = shared + [next(take) for _ in range(cols - len(shared))]
            table.append(row[:cols])
            ctx.append(c)
    return table, ctx, (torch.rand(pool, generator=g) < held).tolist() if held else None


def check_fork(rts, table, ctx, parents, block, pool, held, n_free=None, pad=0):
    want = ref.fork(table, ctx, parents, block, pool, held, pool if n_free is None else n_free)
    got = rts.fork_blocks(padded(table, pad), i32(ctx), i32(parents), block, pool,
                          held=None if held is None else torch.tensor(held, device=DEV), n_free=n_free)
    assert_same(got, want, "fork")
    if rts.raw_library().fork_blocks_workspace_size(len(table), len(table[0]), pool):
        alone = rts.fork_blocks(padded(table, pad), i32(ctx), i32(parents), block, pool, workspace=None,
                                held=None if held is None else torch.tensor(held, device=DEV), n_free=n_free)
        assert all(torch.equal(x, y) for x, y in zip(alone, got))
    return got


@pytest.mark.parametrize("reqs,beams,ctx,block,pool,held,pad", [
    (1, 1, 1, 1, 1, 0, 0), (1, 4, 100, 16, 64, 0, 0), (8, 4, 300, 16, 4096, 0, 3), (8, 4, 300, 16, 700, 0.1, 0),
    (50, 8, 100, 1, 60000, 0, 0), (30, 5, 1000, 24, 9001, 0.05, 1), (512, 8, 200, 128, 30000, 0, 0),
    (4096, 1, 40, 16, 20000, 0.01, 0), (3, 2, 5000, 16, 1 << 19, 0, 0), (3, 2, 50, 16, 33, 0.3, 0),
    (64, 8, 4000, 16, 90000, 0.02, 0), (1500, 2, 2000, 16, 400000, 0, 1), (2, 2, 8000, 1, 50000, 0, 3),
    (4, 4, 9000, 1, 200000, 0.1, 0)])
def test_fork(rts, reqs, beams, ctx, block, pool, held, pad):
    say("fork", reqs, beams, ctx, block, pool, held, pad)
    g = torch.Generator().manual_seed(reqs)
    table, lens, held = setup(reqs, reqs, beams, ctx, block, pool, held)
    rows = reqs * beams
    within = [(i // beams) * beams + int(torch.randint(0, beams, (1,), generator=g)) for i in range(rows)]
    check_fork(rts, table, lens, within, block, pool, held, pad=pad)
    # some end; rows in any order; a number of rows that differs; parents that do not exist
    anywhere = torch.randint(-1, rows + 1, (min(4096, rows // 2 + 3),), generator=g).tolist()
    check_fork(rts, table, lens, anywhere, block, pool, held, n_free=min(pool, 100), pad=pad)
    check_fork(rts, table, lens, [0] * min(9, rows), block, pool, held, n_free=0)


def test_fork_edges(rts):
    # lengths of zero and below, and past the table; entries outside of the pool; whole blocks only
    table = [[5, 6, 7], [1, 99, -3], [2, 3, 4], [8, 9, 10], [5, 6, 0]]
    ctx = [-4, 24, 1000, 32, 20]
    for parents in ([0, 1, 2, 3, 4], [1, 1, 2, 2, 3, 3], [4, 4, 4], [], [2 ** 31 - 1, -2 ** 31, 4]):
        check_fork(rts, table, ctx, parents, 16, 12, None)
        check_fork(rts, table, ctx, parents, 16, 12, [i == 6 for i in range(12)])
        check_fork(rts, table, ctx, parents, 2 ** 31 - 1, 12, None)
    # two parents whose last block is the same; one that is another's whole block
    check_fork(rts, [[0, 1], [2, 1], [3, 1]], [3, 3, 4], [0, 1], 2, 8, None)
    check_fork(rts, [[0, 1], [2, 1], [3, 1]], [3, 3, 4], [2, 1, 1], 2, 8, None)
    check_fork(rts, [[0, 0]], [3], [0], 2, 8, None)
    # a pool that runs out, and one without blocks
    got = check_fork(rts, [[0, 1], [2, 3]], [3, 3], [0, 0, 0, 1, 1], 2, 5, None)
    assert got.counts.tolist() == [0, 3] and got.copies.tolist() == [[1, 4]] + [[-1, -1]] * 4
    check_fork(rts, [[0, 1]], [3], [0, 0], 2, 0, None)
    # no rows, no columns
    got = rts.fork_blocks(torch.empty(0, 4, dtype=torch.int32, device=DEV), i32([]), i32([0, -1]), 16, 3)
    assert got.block_table.tolist() == [[-1] * 4] * 2 and got.free_blocks.tolist() == [0, 1, 2]
    got = rts.fork_blocks(torch.empty(2, 0, dtype=torch.int32, device=DEV), i32([5, 6]), i32([1, 1]), 16, 3)
    assert got.ctx_lens.tolist() == [6, 6] and got.counts.tolist() == [3, 0]


def test_fork_unaligned_held_and_given_outputs(rts):
    table, ctx, held = setup(9, 6, 3, 200, 16, 500, 0.2)
    flags = torch.zeros(600, dtype=torch.uint8, device=DEV)
    for shift in (0, 1, 7):
        part = flags[shift:shift + 500]
        part.copy_(torch.tensor(held, dtype=torch.uint8) * 37)
        parents = [0, 0, 3, 3, 4, 17]
        want = ref.fork(table, ctx, parents, 16, 500, held, 40)
        out = rts.Fork(torch.full((6, len(table[0])), 5, dtype=torch.int32, device=DEV), i32([9] * 6),
                       torch.empty(6, 2, dtype=torch.int32, device=DEV), i32([9] * 40), i32([7, 7]))
        assert_same(rts.fork_blocks(i32(table), i32(ctx), i32(parents), 16, 500, held=part, n_free=40, out=out), want, "")


def check_compact(rts, table, ctx, block, pool, held, max_moves=None, n_free=None, pad=0):
    want = ref.compact(table, ctx, block, pool, held, pool // 2 if max_moves is None else max_moves,
                       pool if n_free is None else n_free)
    got = rts.compact_blocks(padded(table, pad), i32(ctx), block, pool,
                             held=None if held is None else torch.tensor(held, device=DEV), max_moves=max_moves,
                             n_free=n_free)
    assert_same(got, want, "compact")
    if rts.raw_library().compact_blocks_workspace_size(len(table), len(table[0]), pool):
        alone = rts.compact_blocks(padded(table, pad), i32(ctx), block, pool, workspace=None, max_moves=max_moves,
                                   held=None if held is None else torch.tensor(held, device=DEV), n_free=n_free)
        assert all(torch.equal(x, y) for x, y in zip(alone, got))
    return got


@pytest.mark.parametrize("reqs,beams,ctx,block,pool,held,pad", [
    (1, 1, 1, 1, 1, 0, 0), (1, 4, 100, 16, 64, 0, 0), (8, 4, 300, 16, 4096, 0, 3), (8, 4, 300, 16, 700, 0.1, 0),
    (50, 8, 100, 1, 60000, 0, 0), (30, 5, 1000, 24, 9001, 0.05, 1), (5000, 1, 40, 16, 20000, 0.01, 0),
    (3, 2, 5000, 16, 1 << 19, 0.5, 0), (3, 2, 50, 16, 33, 0.3, 0), (64, 8, 4000, 16, 90000, 0.02, 0),
    (1500, 2, 2000, 16, 400000, 0.1, 1), (2, 2, 8000, 1, 50000, 0, 3), (4, 4, 9000, 1, 200000, 0.1, 0)])
def test_compact(rts, reqs, beams, ctx, block, pool, held, pad):
    say("compact", reqs, beams, ctx, block, pool, held, pad)
    table, lens, held = setup(reqs, reqs, beams, ctx, block, pool, held)
    got = check_compact(rts, table, lens, block, pool, held, pad=pad)
    moves = got.counts.tolist()[1]
    check_compact(rts, table, lens, block, pool, held, max_moves=moves // 2, n_free=min(77, pool))
    check_compact(rts, table, lens, block, pool, held, max_moves=0, n_free=0)
    again = got.block_table.tolist()
    assert check_compact(rts, again, lens, block, pool, held).counts.tolist()[1] == 0


def test_compact_edges(rts):
    check_compact(rts, [[5, 6, 7], [1, 99, -3]], [-4, 24], 16, 12, None)
    check_compact(rts, [[11, 10, 9], [9, 8, 11]], [100, 100], 16, 12, [False] * 8 + [True] + [False] * 3)
    check_compact(rts, [[11, 10, 9]], [0], 16, 12, None)           # nothing in use
    check_compact(rts, [[0, 1, 2]], [48], 16, 3, None)             # nothing free
    check_compact(rts, [[0, 1, 2]], [48], 16, 3, [True] * 3)       # nothing may move
    check_compact(rts, [[4, 3, 2]], [48], 16, 5, [True, False, True, False, False])
    check_compact(rts, [[4, 3, 2]], [48], 16, 0, None)
    got = rts.compact_blocks(torch.empty(0, 4, dtype=torch.int32, device=DEV), i32([]), 16, 5)
    assert got.counts.tolist() == [5, 0] and got.free_blocks.tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("block,stride", [(1, 1), (16, 16), (24, 30), (7, 7)])
def test_copy(rts, block, stride):
    """Caches of several types, row lengths and strides, contiguous or not; only the pairs' blocks change."""
    g = torch.Generator().manual_seed(block)
    pool = 50
    rows = pool * stride
    wide = torch.randn(rows, 100, generator=g).to(DEV)
    caches = [torch.randn(rows, 8, 16, generator=g).bfloat16().to(DEV), wide[:, 4:68], wide.bfloat16()[:, 1:34],
              torch.randn(rows, generator=g).to(DEV), torch.randint(0, 256, (rows, 5), generator=g).byte().to(DEV),
              torch.randn(rows, 3, generator=g).bfloat16().to(DEV), torch.randn(rows - 1, 4, generator=g).to(DEV),
              torch.randint(0, 256, (rows * 10 + 7,), generator=g).byte().to(DEV)[7:].view(rows, 10),
              torch.empty(rows, 0, device=DEV), torch.randn(rows + 3, 128, generator=g).to(torch.float8_e4m3fn).to(DEV)]
    ids = torch.randperm(pool, generator=g)[:40].view(20, 2)
    pairs = torch.cat([ids, torch.tensor([[-1, 3], [4, -1], [-1, -1], [pool + 9, 1], [1, pool + 9], [7, 7],
                                          [2 ** 31 - 1, 0], [0, 2 ** 31 - 1], [-2 ** 31, 2]])])
    pairs = pairs[torch.randperm(len(pairs), generator=g)].int().to(DEV)
    want = []
    for c in caches:
        w = c.clone()
        for a, b in pairs.tolist():
            if a >= 0 and b >= 0 and a != b and max(a, b) * stride + block <= c.shape[0]:
                w[b * stride:b * stride + block] = c[a * stride:a * stride + block].clone()
        want.append(w)
    outside = wide.clone()
    rts.copy_blocks(caches, pairs, block, stride_rows=stride)
    torch.cuda.synchronize()
    for i, (c, w) in enumerate(zip(caches, want)):
        same = torch.equal(c.contiguous().view(torch.uint8) if c.numel() else c,
                           w.contiguous().view(torch.uint8) if c.numel() else w)
        assert same, f"cache {i}"
    assert torch.equal(wide[:, :4], outside[:, :4]) and torch.equal(wide[:, 68:], outside[:, 68:])


def test_copy_many_caches_and_none(rts):
    g = torch.Generator().manual_seed(0)
    caches = [torch.randn(64, 24, generator=g).to(DEV) for _ in range(150)]
    before = [c.clone() for c in caches]
    rts.copy_blocks(caches, i32([[0, 3], [2, 1]]), 16)
    for c, b in zip(caches, before):
        assert torch.equal(c[48:], b[:16]) and torch.equal(c[16:32], b[32:48]) and torch.equal(c[32:48], b[32:48])
    rts.copy_blocks(caches[0], i32([[0, 2]]), 16)  # one tensor
    assert torch.equal(caches[0][32:48], before[0][:16])
    rts.copy_blocks([], i32([[0, 1]]), 16)
    rts.copy_blocks(caches, torch.empty(0, 2, dtype=torch.int32, device=DEV), 16)


def test_copy_far_blocks(rts):
    """Blocks past 2^32 bytes, and a block larger than 2^16 words."""
    big = torch.empty(90_000, 32_768, dtype=torch.bfloat16, device=DEV)
    big[:300] = 1.0
    big[89_700:] = 2.0
    rts.copy_blocks([big], i32([[0, 150], [299, 3]]), 300)
    assert bool((big[45_000:45_300] == 1).all()) and bool((big[900:1200] == 2).all())


def test_block_calls_captured(rts):
    """A captured fork, its copies and a compaction, replayed on other inputs, against eager calls."""
    pool, block = 300, 16
    cache = torch.randn(pool * block, 8, device=DEV)
    table, ctx, _ = setup(1, 5, 4, 120, block, pool, 0)
    t, c, p = i32(table), i32(ctx), i32([0] * 20)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = rts.fork_blocks(t, c, p, block, pool)
        rts.copy_blocks([cache], f.copies, block)
        m = rts.compact_blocks(f.block_table, f.ctx_lens, block, pool)
    for seed in (2, 3, 4):
        table, ctx, _ = setup(seed, 5, 4, 120, block, pool, 0)
        parents = torch.randint(-1, 20, (20,), generator=torch.Generator().manual_seed(seed)).tolist()
        t.copy_(torch.tensor(table))
        c.copy_(torch.tensor(ctx))
        p.copy_(torch.tensor(parents))
        before = cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.fork(table, ctx, parents, block, pool, None, pool)
        assert_same(f, want, "fork")
        assert_same(m, ref.compact(want["block_table"], want["ctx_lens"], block, pool, None, pool // 2, pool), "compact")
        for a, b in want["copies"]:
            if a >= 0:
                before[b * block:(b + 1) * block] = before[a * block:(a + 1) * block]
        assert torch.equal(cache, before)


def test_streams(rts):
    """Calls on another stream take their memory from it, behind work that keeps the current stream busy."""
    pool, block = 400, 16
    table, ctx, _ = setup(6, 40, 4, 120, block, pool, 0)
    parents = list(range(160))
    cache = torch.randn(pool * block, 8, device=DEV)
    before = cache.clone()
    t, c, p = i32(table), i32(ctx), i32([x // 2 for x in parents])
    want = ref.fork(table, ctx, p.tolist(), block, pool, None, pool)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        junk = torch.full((200_000,), 7, dtype=torch.int32, device=DEV)
        torch.cuda._sleep(10_000_000)
        junk.fill_(9)
        del junk  # given back to the current stream, which is still to write it
        f = rts.fork_blocks(t, c, p, block, pool, stream=side)
        m = rts.compact_blocks(t, c, block, pool, stream=side)
        rts.copy_blocks([cache], f.copies, block, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert_same(f, want, "fork")
        assert_same(m, ref.compact(table, ctx, block, pool, None, pool // 2, pool), "compact")
    for a, b in want["copies"]:
        if a >= 0:
            before[b * block:(b + 1) * block] = before[a * block:(a + 1) * block]
    assert torch.equal(cache, before)


def test_large_tables_captured_and_at_once(rts):
    """Tables that several workgroups read first: replays on other inputs, and calls at the same time."""
    pool, block, rows = 90_000, 16, 400
    assert rts.raw_library().fork_blocks_workspace_size(rows, 251, pool) > 0
    cases = []
    for seed in (21, 22, 23):
        table, ctx, held = setup(seed, 50, 8, 4000, block, pool, 0.02)
        parents = torch.randint(-1, rows, (rows,), generator=torch.Generator().manual_seed(seed)).tolist()
        assert len(table) == rows and len(table[0]) == 251
        cases.append((table, ctx, held, parents, ref.fork(table, ctx, parents, block, pool, held, pool),
                      ref.compact(table, ctx, block, pool, held, pool // 2, pool)))
    t, c, p = i32(cases[0][0]), i32(cases[0][1]), i32(cases[0][3])
    h = torch.tensor(cases[0][2], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = rts.fork_blocks(t, c, p, block, pool, held=h)
        m = rts.compact_blocks(t, c, block, pool, held=h)
    for table, ctx, held, parents, forked, compacted in cases:
        t.copy_(torch.tensor(table))
        c.copy_(torch.tensor(ctx))
        p.copy_(torch.tensor(parents))
        h.copy_(torch.tensor(held))
        graph.replay()
        torch.cuda.synchronize()
        assert_same(f, forked, "fork")
        assert_same(m, compacted, "compact")
    streams = [torch.cuda.Stream() for _ in cases]
    inputs = [(i32(x[0]), i32(x[1]), i32(x[3]), torch.tensor(x[2], device=DEV)) for x in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [(rts.fork_blocks(t, c, p, block, pool, held=h, stream=s), rts.compact_blocks(t, c, block, pool, held=h, stream=s))
               for s, (t, c, p, h) in zip(streams, inputs)]
        torch.cuda.synchronize()
        for (f, m), x in zip(got, cases):
            assert_same(f, x[4], "fork")
            assert_same(m, x[5], "compact")
