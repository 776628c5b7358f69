"""Calls with ``stream=``: what a call allocates must not be memory that the current
stream has given back but is still to use, and results may be read on the
current stream after it has waited for the call's."""

import pytest

from gpu_common import say

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"
SPIN = 100_000_000  # clock ticks that the current stream is kept busy for


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def calls(rts):
    """{name: a call that allocates its outputs (and a workspace where it takes one)}."""
    g = torch.Generator().manual_seed(0)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    long = i32([200, 100, 250])
    ctx, new, free = i32([40, 3, 0]), i32([1, 2, 5]), torch.arange(100, 140, dtype=torch.int32, device=DEV)
    table = torch.randperm(60, generator=g).int().view(3, 20).to(DEV)
    scratch_table = table.clone()
    q_i, keys, w = rand(8, 32, 128), rand(960, 128), rand(8, 32, dtype=torch.float32)
    req, ends = i32([0, 1, 1, 2, 2, 2, 2, 2]), i32([300] * 8)
    q, cache = rand(8, 16, 576), rand(960, 576)
    ids = torch.randint(0, 960, (8, 900), generator=g).int().to(DEV)
    starts = i32([0, 1, 3, 8])
    parts, lse = rand(3, 8, 16, 512), rand(3, 8, 16, dtype=torch.float32)
    wide = rand(2, 300_000, dtype=torch.float32)
    local = rand(4, 2000)
    local_ids = rts.topk_rows(local, 64)
    packed = torch.stack([rts.pack_candidates(local, local_ids) for _ in range(2)])
    pairs = torch.stack([rts.pack_pairs(local.float(), local_ids, r, 2) for r in range(2)])
    r4, scores = i32([0, 1, 2, 0]), local.float()
    packed_rows = packed.transpose(0, 1).contiguous()
    pair_rows = pairs.transpose(0, 1).contiguous().view(4, 128, 2)
    return {
        "assign_slots": lambda s: tuple(rts.assign_slots(ctx, new, 11, scratch_table, free, 16, stream=s)),
        "indexer_logits": lambda s: rts.indexer_logits(q_i, keys, w, stream=s),
        "indexer_logits_paged": lambda s: rts.indexer_logits_paged(
            q_i, keys, w, req, ends, table, 16, 300, stream=s),
        "latent_attend_rows": lambda s: rts.latent_attend_rows(q, cache, ids, 0.07, stream=s),
        "latent_attend_paged": lambda s: rts.latent_attend_paged(q, cache, starts, long, table, 16, 0.07, stream=s),
        "merge_attend_rank_major": lambda s: rts.merge_attend_rank_major(parts, lse, stream=s),
        "topk_rows": lambda s: rts.topk_rows(wide, 512, stream=s),
        "pack_candidates": lambda s: rts.pack_candidates(local, local_ids, stream=s),
        "pack_pairs": lambda s: rts.pack_pairs(scores, local_ids, 0, 2, stream=s),
        "merge_select_rank_major": lambda s: rts.merge_select_rank_major(packed, 64, stream=s),
        "merge_select_row_major": lambda s: rts.merge_select_row_major(packed_rows, 64, stream=s),
        "merge_select_pairs_rank_major": lambda s: rts.merge_select_pairs_rank_major(pairs, 64, stream=s),
        "merge_select_pairs_row_major": lambda s: rts.merge_select_pairs_row_major(pair_rows, 64, 2, stream=s),
        "emit_rows": lambda s: rts.emit_rows(local_ids, 2, 1, r4, table, 16, 16, stream=s),
        "merge_select_rank_major_rows": lambda s: rts.merge_select_rank_major_rows(
            packed, 64, 1, r4, table, 16, 16, stream=s)[:2],
    }


NAMES = ["assign_slots", "indexer_logits", "indexer_logits_paged", "latent_attend_rows", "latent_attend_paged",
         "merge_attend_rank_major", "topk_rows", "pack_candidates", "pack_pairs", "merge_select_rank_major",
         "merge_select_row_major", "merge_select_pairs_rank_major", "merge_select_pairs_row_major", "emit_rows",
         "merge_select_rank_major_rows"]


def flat(x):
    return [t for t in (x if isinstance(x, tuple) else (x,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_of_a_call_on_another_stream(rts, name, monkeypatch):
    """The current stream is busy, and what it has queued behind that still writes to memory of the call's
    sizes that was given back already; the call on the side stream runs meanwhile."""
    say("allocations on another stream:", name)
    call = calls(rts)[name]
    empty, made = torch.empty, []

    def spy(*a, **kw):
        t = empty(*a, **kw)
        if t.is_cuda:
            made.append((t.data_ptr(), t.numel() * t.element_size()))
        return t

    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", spy)
        call(None)                       # how much it allocates
    sizes = [n for _, n in made if n]
    assert sizes
    torch.cuda.synchronize()

    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SPIN)
    pending = set()
    for n in sizes * 2:
        t = empty(n, dtype=torch.uint8, device=DEV)
        t.fill_(0x55)
        pending.add(t.data_ptr())
        del t                            # given back while the fill is still queued
    made.clear()
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", spy)
        got = flat(call(side))
    assert made and not pending & {p for p, n in made if n}, "memory that the current stream still writes to"
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_split_calls_on_two_streams_share_no_workspace(rts):
    """One call on the current stream and one on another at once, many times: both split their lists."""
    say("a call on the current stream beside one on another")
    g = torch.Generator().manual_seed(1)
    q = torch.randn(4, 32, 576, generator=g).bfloat16().to(DEV)
    cache = torch.randn(3000, 576, generator=g).bfloat16().to(DEV)
    lists = [torch.randint(0, 3000, (4, 1500), generator=g).int().to(DEV) for _ in range(2)]
    assert rts.latent_attend_rows_workspace_size(4, 32, 512, 1500) > 0
    want = [rts.latent_attend_rows(q, cache, ids, 0.07) for ids in lists]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        got[0].append(rts.latent_attend_rows(q, cache, lists[0], 0.07))
        got[1].append(rts.latent_attend_rows(q, cache, lists[1], 0.07, stream=side))
    torch.cuda.synchronize()
    for k in range(2):
        for o, l in got[k]:
            assert torch.equal(o, want[k][0]) and torch.equal(l, want[k][1])


def test_results_read_on_the_current_stream_are_kept_for_it(rts):
    """A result of a side-stream call that the current stream still reads when it is dropped is not handed
    to the side stream's next call."""
    say("a dropped result that the current stream still reads")
    parts = [torch.full((2, 64, 16, 512), float(v), dtype=torch.bfloat16, device=DEV) for v in (3, 5)]
    lse = torch.zeros(2, 64, 16, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first, _ = rts.merge_attend_rank_major(parts[0], lse, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SPIN)
    copy = first.clone()                 # queued behind the spin
    del first
    later = [rts.merge_attend_rank_major(parts[1], lse, stream=side)[0] for _ in range(3)]
    torch.cuda.synchronize()
    assert (copy == 3).all() and all((x == 5).all() for x in later)


@pytest.mark.parametrize("name", ["assign_slots", "indexer_logits_paged", "latent_attend_rows", "latent_attend_paged",
                                  "merge_attend_rank_major", "topk_rows"])
def test_captured_beside_a_call_on_another_stream(rts, name):
    """A graph with the same call on its own stream and on one that joins it, replayed with eager calls between."""
    say("captured on two streams:", name)
    call = calls(rts)[name]
    want = [t.clone() for t in flat(call(None))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        on_side = flat(call(side))
        if name != "assign_slots":       # which writes one table
            here = flat(call(None))
        torch.cuda.current_stream().wait_stream(side)
        if name == "assign_slots":
            here = flat(call(None))
    for _ in range(4):
        for t in on_side + here:
            t.view(torch.uint8).fill_(0x33)
        graph.replay()
        eager = flat(call(None))
        torch.cuda.synchronize()
        for x, y, z, w in zip(on_side, here, eager, want):
            assert all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t in (x, y, z))
