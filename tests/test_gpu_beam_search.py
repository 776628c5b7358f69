"""A beam search over a paged cache, as a serving loop runs it: selection, forked and
freed blocks, their copies, slots of the new tokens, attention, from time to time a
compaction.  Every stage of every step is checked against plain implementations that
know each hypothesis by its list of tokens and no pages."""

import math
from types import SimpleNamespace

import pytest

import beam_reference as ref
from gpu_common import say
from serving_reference import assert_close

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def rts():
    import row_top_select_amd
    return row_top_select_amd


class Model:
    """One layer of attention: keys, values and queries by token and position, logits from the heads' outputs."""

    def __init__(self, seed, vocab, heads, kv, dim, longest):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv, self.dim, self.vocab, self.scale = heads, kv, dim, vocab, dim ** -0.5
        rand = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)  # noqa: E731
        self.k, self.v, self.q = rand(vocab, kv, dim), rand(vocab, kv, dim), rand(vocab, heads, dim)
        self.pos = rand(longest, 1, dim)
        self.head = torch.randn(heads * dim, vocab, generator=g).to(DEV) * 4 * (heads * dim) ** -0.5

    def kv_of(self, tokens, pos):
        return self.k[tokens] + self.pos[pos], self.v[tokens] - self.pos[pos]

    def q_of(self, tokens, pos):
        return self.q[tokens] + self.pos[pos]

    def logits(self, out):
        return out.float().view(out.shape[0], -1) @ self.head


def start(model, prompts, beams, block, pool, cols):
    """The state behind the prompts: one live beam a request, whose blocks are filled; the others are empty rows."""
    rows = len(prompts) * beams
    table = torch.full((rows, cols), -1, dtype=torch.int32, device=DEV)
    ctx = torch.zeros(rows, dtype=torch.int32, device=DEV)
    k = torch.full((pool * block + 1, model.kv, model.dim), math.nan, dtype=torch.bfloat16, device=DEV)
    v = torch.full_like(k, math.nan)
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(1)).tolist()
    logits = torch.zeros(rows, model.vocab, device=DEV)
    scores = torch.full((len(prompts), beams), -math.inf, device=DEV)
    for r, prompt in enumerate(prompts):
        row, n = r * beams, len(prompt)
        mine = [order.pop() for _ in range(-(-n // block))]
        table[row, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
        at = torch.tensor([mine[p // block] * block + p % block for p in range(n)], device=DEV)
        t, p = torch.tensor(prompt, device=DEV), torch.arange(n, device=DEV)
        k[at], v[at] = model.kv_of(t, p)
        ctx[row] = n
        kk, vv = model.kv_of(t, p)
        z = torch.einsum("hgd,nhd->hgn", model.q_of(t[-1:], p[-1:])[0].float().view(model.kv, -1, model.dim), kk.float())
        out = torch.einsum("hgn,nhd->hgd", torch.softmax(z * model.scale, 2), vv.float())
        logits[row] = model.logits(out.reshape(1, model.heads, model.dim).bfloat16())[0]
        scores[r, 0] = 0
    return SimpleNamespace(table=table, ctx=ctx, k=k, v=v, logits=logits, scores=scores,
                           done=torch.zeros(rows, dtype=torch.bool, device=DEV))


def step(rts, model, st, beams, block, pool, eos):
    """One step; the state's tensors are written in place, so that it can be captured."""
    picked = rts.beam_select(st.logits, st.scores, beams, eos=eos)
    parents = torch.where(st.done, -1, picked.parents.view(-1))
    f = rts.fork_blocks(st.table, st.ctx, parents, block, pool)
    rts.copy_blocks([st.k, st.v], f.copies, block)
    m = rts.assign_slots(f.ctx_lens, (parents >= 0).int(), parents.numel(), f.block_table, f.free_blocks, block)
    live = m.req_id >= 0
    row = m.req_id.clamp(min=0).long()
    tokens = picked.tokens.view(-1)[row].clamp(min=0).long()
    pos = (m.row_ends - 1).clamp(min=0).long()
    slots = torch.where(m.slots >= 0, m.slots, st.k.shape[0] - 1).long()
    knew, vnew = model.kv_of(tokens, pos)
    st.k.index_copy_(0, slots, knew)
    st.v.index_copy_(0, slots, vnew)
    out, lse = rts.kv_attend_paged(model.q_of(tokens, pos), st.k, st.v, m.req_id, m.row_ends, f.block_table, block,
                                   model.scale)
    logits = torch.zeros_like(st.logits).index_add_(0, row, model.logits(out) * live[:, None])
    st.table.copy_(f.block_table)
    st.ctx.copy_(f.ctx_lens + (parents >= 0).int())
    scores = torch.where((parents >= 0).view(st.scores.shape), picked.scores, -math.inf)
    result = SimpleNamespace(picked=picked, parents=parents, fork=f, slots=m, out=out, lse=lse, logits=st.logits.clone(),
                             old_scores=st.scores.clone())
    st.logits.copy_(logits)
    st.scores.copy_(scores)
    return result


def check_step(model, r, hypotheses, table, ctx, beams, block, pool, eos, what):
    """The stages of a step by the hypotheses before it (lists of tokens by row, None: an empty row); returns those after it."""
    check = SimpleNamespace(scores=r.picked.scores, parents=r.picked.parents, tokens=r.picked.tokens, ended=r.picked.ended)
    ref.check_beams(check, r.logits.cpu(), r.old_scores.cpu(), beams, eos, what)
    parents, tokens = r.parents.tolist(), r.picked.tokens.view(-1).tolist()
    want = ref.fork(table, ctx, parents, block, pool, None, pool)
    assert r.fork.copies.tolist() == want["copies"] and r.fork.ctx_lens.tolist() == want["ctx_lens"], what
    assert r.fork.counts.tolist() == want["counts"] and r.fork.free_blocks.tolist() == want["free_blocks"], what
    assert want["counts"][0] >= 0 and all(p < 0 or hypotheses[p] is not None for p in parents), what
    after = [None if p < 0 else hypotheses[p] + [t] for p, t in zip(parents, tokens)]
    req = r.slots.req_id.tolist()
    got, lse, ob, lb, wo, wl = r.out.cpu(), r.lse.cpu(), [], [], [], []
    for i, row in enumerate(req):
        h = after[row] if row >= 0 else []
        t = torch.tensor(h, dtype=torch.long, device=DEV)
        p = torch.arange(len(h), device=DEV)
        k, v = (x.cpu().float() for x in model.kv_of(t, p))
        q = model.q_of(t[-1:], p[-1:]).cpu()[0] if h else torch.zeros(model.heads, model.dim)
        for j in range(model.kv):
            n = model.heads // model.kv
            for a, b in zip((wo, wl, ob, lb), ref.kv_attend(q[j * n:(j + 1) * n], k[:, j], v[:, j], model.scale)):
                a.append(b)
    shape = (len(req), model.heads)
    assert_close(got, torch.stack(wo).view(*shape, model.dim), torch.stack(ob).view(*shape, model.dim), what)
    assert_close(lse, torch.stack(wl).view(shape), torch.stack(lb).view(shape), what)
    return after


@pytest.mark.parametrize("beams,block,heads,kv,dim", [(3, 4, 4, 2, 64), (4, 16, 8, 1, 128), (1, 5, 2, 2, 64)])
def test_beam_search(rts, beams, block, heads, kv, dim):
    say("beam search", beams, block, heads, kv, dim)
    eos, vocab = 5, 211
    g = torch.Generator().manual_seed(beams)
    prompts = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in (7, 1, 33, 16, 12)]
    rows, cols = len(prompts) * beams, -(-60 // block)
    pool = rows * cols // 2 + 3
    model = Model(beams, vocab, heads, kv, dim, 64)
    st = start(model, prompts, beams, block, pool, cols)
    hypotheses = [prompts[r // beams] if r % beams == 0 else None for r in range(rows)]
    for n in range(14):
        table, ctx = st.table.tolist(), st.ctx.tolist()
        r = step(rts, model, st, beams, block, pool, eos)
        hypotheses = check_step(model, r, hypotheses, table, ctx, beams, block, pool, eos, f"step {n}")
        if n == 5:  # the second request ends: its blocks become free
            st.done[beams:2 * beams] = True
        if n in (3, 9):
            # The pool's live blocks move to its front; the search goes on over them.
            m = rts.compact_blocks(st.table, st.ctx, block, pool)
            want = ref.compact(st.table.tolist(), st.ctx.tolist(), block, pool, None, pool // 2, pool)
            assert m.block_table.tolist() == want["block_table"] and m.counts.tolist() == want["counts"]
            rts.copy_blocks([st.k, st.v], m.moves, block)
            st.table.copy_(m.block_table)
            used = {i for row, c in zip(st.table.tolist(), st.ctx.tolist()) for i in row[:-(-c // block)]}
            assert used == set(range(len(used)))
            gone = torch.ones(pool, dtype=torch.bool, device=DEV)
            gone[list(used)] = False
            st.k[:-1].view(pool, -1)[gone] = math.nan  # nothing of them is read any more
            st.v[:-1].view(pool, -1)[gone] = math.nan
    assert st.ctx.tolist()[beams] == 0 and all(h is None for h in hypotheses[beams:2 * beams])


def test_captured_beam_search(rts):
    """The same step in a graph, replayed with eager work in between."""
    eos, vocab, beams, block = 3, 97, 3, 4
    g = torch.Generator().manual_seed(9)
    prompts = [torch.randint(0, vocab, (n,), generator=g).tolist() for n in (5, 9)]
    rows, cols, pool = len(prompts) * beams, 12, 70
    model = Model(11, vocab, 4, 2, 64, 64)
    st = start(model, prompts, beams, block, pool, cols)
    saved = {n: t.clone() for n, t in vars(st).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(rts, model, st, beams, block, pool, eos)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step(rts, model, st, beams, block, pool, eos)
    for n, t in saved.items():
        getattr(st, n).copy_(t)
    hypotheses = [prompts[i // beams] if i % beams == 0 else None for i in range(rows)]
    for n in range(8):
        table, ctx = st.table.tolist(), st.ctx.tolist()
        graph.replay()
        torch.cuda.synchronize()
        hypotheses = check_step(model, r, hypotheses, table, ctx, beams, block, pool, eos, f"replay {n}")
