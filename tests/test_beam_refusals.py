"""Refusals of the operators of a beam-search step: the C ABI rejects bad arguments on the
host and the binding rejects bad tensors (no kernel runs in these tests)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import row_top_select_amd as rts  # noqa: E402

EINVAL, EUNSUP, EWS = -1, -2, -3
P = ctypes.c_void_p(0x10000)     # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x10001)
lib = rts.raw_library()


def beam(**kw):
    a = dict(logits=P, dtype=0, groups=2, beams=4, vocab=100000, ld=100000, scores=P, k=4, eos=2, out=P, parents=P, tokens=P,
             ended=P, ws=P, ws_bytes=1 << 20)
    a.update(kw)
    return lib.beam_select(*a.values(), None)


def test_beam_select():
    for kw in (dict(dtype=2), dict(groups=-1), dict(beams=0), dict(vocab=0), dict(ld=99999), dict(k=0), dict(eos=-2),
               dict(eos=100000), dict(eos=-1), dict(ended=None), dict(logits=None), dict(scores=None), dict(out=None),
               dict(parents=None), dict(tokens=None), dict(ws=None), dict(logits=ODD), dict(scores=ODD), dict(out=ODD),
               dict(parents=ODD), dict(tokens=ODD), dict(ended=ODD), dict(ws=ODD), dict(dtype=1, logits=ODD)):
        assert beam(**kw) == EINVAL, kw
    for kw in (dict(beams=65), dict(k=65), dict(vocab=1 << 31, ld=1 << 31), dict(groups=1 << 30)):
        assert beam(**kw) == EUNSUP, kw
    assert beam(groups=0) == 0
    need = lib.beam_select_workspace_size(0, 2, 4, 100000, 4)
    assert need > 0 and beam(ws_bytes=need - 1) == EWS
    assert lib.beam_select_workspace_size(0, 2, 4, 1000, 4) == 0 and beam(vocab=1000, ws=None) == EINVAL  # but a size
    for bad in ((2, 2, 4, 1000, 4), (0, 0, 4, 1000, 4), (0, 2, 65, 1000, 4), (0, 2, 4, 0, 4), (0, 2, 4, 1000, 65)):
        assert lib.beam_select_workspace_size(*bad) == 0, bad


def fork(**kw):
    a = dict(table=P, rows_in=4, cols=8, ld=8, ctx=P, parents=P, rows_out=4, block=16, pool=100, held=P, out=P, ld_out=8,
             lens=P, copies=P, free=P, n_free=10, counts=P, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.fork_blocks(*a.values(), None)


def test_fork_blocks():
    for kw in (dict(rows_in=-1), dict(cols=-1), dict(ld=7), dict(rows_out=-1), dict(block=0), dict(pool=-1),
               dict(ld_out=7), dict(n_free=-1)):
        assert fork(**kw) == EINVAL, kw
    for name in ("table", "ctx", "parents", "out", "lens", "copies", "free", "counts"):
        assert fork(**{name: None}) == EINVAL and fork(**{name: ODD}) == EINVAL, name
    assert fork(copies=ctypes.c_void_p(0x10004)) == EINVAL
    for kw in (dict(rows_in=4097), dict(rows_out=4097), dict(pool=(1 << 19) + 1)):
        assert fork(**kw) == EUNSUP, kw
    assert fork(ws_bytes=4) == EINVAL and fork(ws=ODD, ws_bytes=4) == EINVAL
    size = lib.fork_blocks_workspace_size
    assert size(4, 8, 100) == 0 and size(4097, 8, 100) == 0 and size(4096, 800, (1 << 19) + 1) == 0
    need = size(4096, 800, 5000)
    assert need > 0 and fork(rows_in=4096, cols=800, ld=800, ld_out=800, pool=5000, ws=P, ws_bytes=need - 4) == EWS


def compact(**kw):
    a = dict(table=P, rows=4, cols=8, ld=8, ctx=P, block=16, pool=100, held=P, out=P, ld_out=8, moves=P, max_moves=50,
             free=P, n_free=10, counts=P, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.compact_blocks(*a.values(), None)


def test_compact_blocks():
    for kw in (dict(rows=-1), dict(cols=-1), dict(ld=7), dict(block=0), dict(pool=-1), dict(ld_out=7),
               dict(max_moves=-1), dict(n_free=-1)):
        assert compact(**kw) == EINVAL, kw
    for name in ("table", "ctx", "out", "moves", "free", "counts"):
        assert compact(**{name: None}) == EINVAL and compact(**{name: ODD}) == EINVAL, name
    assert compact(moves=ctypes.c_void_p(0x10004)) == EINVAL
    for kw in (dict(rows=1 << 31), dict(pool=(1 << 19) + 1)):
        assert compact(**kw) == EUNSUP, kw
    assert compact(ws_bytes=4) == EINVAL and compact(ws=ODD, ws_bytes=4) == EINVAL
    size = lib.compact_blocks_workspace_size
    assert size(4, 8, 100) == 0 and size(1 << 31, 8, 100) == 0 and size(4096, 800, (1 << 19) + 1) == 0
    need = size(10000, 800, 5000)
    assert need > 0 and compact(rows=10000, cols=800, ld=800, ld_out=800, pool=5000, ws=P, ws_bytes=need - 4) == EWS


def copy(caches=((0x10000, 64, 32, 32),), **kw):
    array = (rts._Cache * max(1, len(caches)))(*caches)
    a = dict(caches=array, n=len(caches), pairs=P, n_pairs=3, block=16, stride=16)
    a.update(kw)
    return lib.copy_blocks(*a.values(), None)


def test_copy_blocks():
    for kw in (dict(caches=((0x10000, -1, 32, 32),)), dict(caches=((0x10000, 64, 0, 32),)),
               dict(caches=((0x10000, 64, 33, 32),)), dict(caches=((None, 64, 32, 32),)), dict(n=-1), dict(pairs=None),
               dict(pairs=ctypes.c_void_p(0x10004)), dict(n_pairs=-1), dict(block=0), dict(stride=-1)):
        assert copy(**kw) == EINVAL, kw
    assert lib.copy_blocks(None, 1, P, 3, 16, 16, None) == EINVAL
    for kw in (dict(caches=((0x10000, 64, 32, 32),) * 65), dict(n_pairs=1 << 31),
               dict(caches=((0x10000, 1 << 31, 32, 32),)), dict(caches=((0x10000, 64, 1 << 31, 1 << 31),)),
               dict(caches=((0x10000, 64, 32, 1 << 31),))):
        assert copy(**kw) == EUNSUP, kw
    assert copy(n_pairs=0) == 0 and copy(caches=()) == 0
    assert copy(caches=((0x10000, 15, 32, 32), (None, 0, 32, 32))) == 0  # no block lies in them


def attend(**kw):
    a = dict(q=P, rows=4, heads=16, ld_q=2048, ld_qhead=128, k=P, v=P, dtype=1, kv=4, dim=128, cache_rows=64, ld_cache=512,
             ld_head=128, ks=P, vs=P, req=P, ends=P, table=P, t_rows=2, t_cols=4, ld_t=4, block=16, stride=16, window=0,
             max_len=64, scale=0.1, out=P, lse=P, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.kv_attend_paged(*a.values(), None)


def test_kv_attend_paged():
    for kw in (dict(dtype=0), dict(rows=-1), dict(heads=0), dict(kv=0), dict(kv=3), dict(dim=0), dict(cache_rows=-1),
               dict(window=-1), dict(max_len=-1), dict(ld_q=-8), dict(ld_qhead=127), dict(ld_cache=-8), dict(ld_head=127),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=-1.8e38), dict(q=None), dict(k=None),
               dict(v=None), dict(out=None), dict(req=None), dict(ends=None), dict(table=None), dict(t_rows=-1),
               dict(t_cols=-1), dict(ld_t=3), dict(block=0), dict(stride=-1), dict(ws_bytes=4), dict(ld_q=2052),
               dict(ld_qhead=132), dict(ld_cache=516), dict(ld_head=132), dict(dtype=2, ld_cache=520),
               dict(dtype=2, ld_head=136)):
        assert attend(**kw) == EINVAL, kw
    for name in ("q", "k", "v", "ks", "vs", "req", "ends", "table", "out", "lse"):
        assert attend(**{name: ODD}) == EINVAL, name
    for kw in (dict(dim=96, ld_qhead=96, ld_head=96), dict(heads=1028), dict(rows=1 << 28), dict(cache_rows=1 << 31),
               dict(ld_cache=(1 << 30) + 8), dict(t_rows=1 << 31)):
        assert attend(**kw) == EUNSUP, kw
    assert attend(rows=0) == 0
    size = lib.kv_attend_paged_workspace_size
    need = size(1, 16, 4, 128, 1, 8192, 0)
    assert need > 0 and size(1, 16, 4, 128, 1, 8192, 64) == 0  # a window of one piece
    assert attend(rows=1, max_len=8192, ws=P, ws_bytes=need - 16) == EWS
    assert attend(rows=1, max_len=8192, ws=ctypes.c_void_p(0x10004), ws_bytes=need) == EINVAL
    for bad in ((0, 16, 4, 128, 1, 64, 0), (1, 16, 3, 128, 1, 64, 0), (1, 16, 4, 96, 1, 64, 0), (1, 16, 4, 128, 0, 64, 0),
                (1, 16, 4, 128, 1, -1, 0), (1, 16, 4, 128, 1, 64, -1), (1, 1028, 4, 128, 1, 64, 0)):
        assert size(*bad) == 0, bad


def test_kv_attend_paged_plan():
    i64 = ctypes.c_int64
    p = (i64 * 2)()
    f = lambda rows=4, heads=16, kv=4, dim=128, dt=1, n=4096, w=0, split=1, plan=p: lib.kv_attend_paged_plan(  # noqa: E731
        i64(rows), heads, kv, dim, dt, i64(n), i64(w), split, plan)
    for kw in (dict(rows=0), dict(heads=0), dict(kv=0), dict(kv=3), dict(dt=0), dict(n=-1), dict(w=-1), dict(plan=None)):
        assert f(**kw) == EINVAL, kw
    for kw in (dict(heads=1028), dict(dim=96), dict(rows=1 << 31)):
        assert f(**kw) == EUNSUP, kw
    assert f(split=0) == 0 and p[0] == 0
    assert f() == 0 and p[0] > 1 and p[1] >= 32
    assert f(w=64) == 0 and p[0] == 0


def test_outputs_in_place():
    other = ctypes.c_void_p(0x20000)
    assert beam(k=5) == EINVAL  # scores of 4 beams, 5 picks
    assert fork(lens=other) == EINVAL and fork(out=other) == EINVAL
    assert fork(out=other, lens=other, parents=other) == EINVAL
    assert compact() == EINVAL


def test_binding():
    z = torch.zeros
    i = dict(dtype=torch.int32)
    b = dict(dtype=torch.bfloat16)
    for call in (lambda: rts.beam_select(z(4, 10), z(1, 4), 2), lambda: rts.fork_blocks(z(2, 3, **i), z(2, **i), z(2, **i), 16, 9),
                 lambda: rts.compact_blocks(z(2, 3, **i), z(2, **i), 16, 9),
                 lambda: rts.copy_blocks([z(32, 4)], z(1, 2, **i), 16),
                 lambda: rts.kv_attend_paged(z(2, 4, 64, **b), z(9, 2, 64, **b), z(9, 2, 64, **b), z(2, **i), z(2, **i),
                                             z(2, 1, **i), 2, 0.1)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_inputs_that_require_gradients_are_refused():
    z = torch.zeros
    i, b = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    x, s = z(4, 10), z(1, 4)
    q, k, v, ks = z(2, 4, 64, **b), z(9, 2, 64, **b), z(9, 2, 64, **b), z(2)
    for call, inputs in ((lambda: rts.beam_select(x, s, 2), (x, s)),
                         (lambda: rts.kv_attend_paged(q, k, v, z(2, **i), z(2, **i), z(2, 1, **i), 2, 0.1, k_scales=ks),
                          (q, k, v, ks))):
        for t in inputs:
            t.requires_grad_(True)
            with pytest.raises(ValueError, match="backward"):
                call()
            t.requires_grad_(False)
