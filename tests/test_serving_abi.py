"""Refusals of the serving-path entry points: the C ABI rejects bad arguments on
the host and the binding rejects bad tensors (no kernel runs in these tests)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import row_top_select_amd as rts  # noqa: E402

EINVAL, EUNSUP, EWS = -1, -2, -3
P = ctypes.c_void_p(0x10000)     # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(0x10002)
lib = rts.raw_library()


def slots(**kw):
    a = dict(ctx=P, new=P, reqs=4, tokens=8, block=16, stride=16, free=P, n=4, table=P, cols=4, ld=4, starts=P,
             req=P, ends=P, slots=P, used=P)
    a.update(kw)
    return lib.assign_slots(*a.values(), None)


def test_assign_slots_refusals():
    assert slots(reqs=-1) == EINVAL and slots(tokens=-1) == EINVAL and slots(block=0) == EINVAL
    assert slots(stride=-1) == EINVAL and slots(n=-1) == EINVAL and slots(ld=3) == EINVAL
    assert slots(cols=-1) == EINVAL
    for name in ("ctx", "new", "free", "table", "starts", "req", "ends", "slots", "used"):
        assert slots(**{name: None}) == EINVAL, name
        assert slots(**{name: ODD}) == EINVAL, name
    assert slots(reqs=8193) == EUNSUP and slots(tokens=1 << 31) == EUNSUP and slots(n=1 << 31) == EUNSUP


def logits(paged=False, **kw):
    a = dict(q=P, dtype=1, rows=4, heads=8, dim=128, ld_q=1024, keys=P)
    if paged:
        a["cache_rows"] = 64
    else:
        a["cols"] = 64
    a.update(ld_keys=128, w=P, ld_w=8, ks=P)
    if paged:
        a.update(req=P, ends=P, table=P, t_rows=2, t_cols=4, ld_t=4, block=16, stride=16, cols=64)
    else:
        a.update(ends=P)
    a.update(out=P, odt=0, ld_out=64)
    a.update(kw)
    return (lib.indexer_logits_paged if paged else lib.indexer_logits)(*a.values(), None)


@pytest.mark.parametrize("paged", [False, True])
def test_indexer_logits_refusals(paged):
    for kw in (dict(dtype=0), dict(dtype=3), dict(odt=2), dict(rows=-1), dict(cols=-1), dict(heads=0), dict(dim=0),
               dict(ld_q=1023), dict(ld_keys=127), dict(ld_w=7), dict(ld_out=63), dict(q=None), dict(keys=None),
               dict(w=None), dict(out=None), dict(q=ODD), dict(keys=ODD), dict(w=ODD), dict(ks=ODD), dict(ends=ODD),
               dict(out=ODD), dict(ld_q=1028), dict(ld_keys=132)):
        assert logits(paged, **kw) == EINVAL, kw
    for kw in (dict(heads=129, ld_q=129 * 128, ld_w=129), dict(dim=96), dict(dim=256, ld_q=2048, ld_keys=256),
               dict(cols=1 << 31, ld_out=1 << 31), dict(ld_keys=(1 << 30) + 16)):
        assert logits(paged, **kw) == EUNSUP, kw
    assert logits(paged, rows=0) == 0 and logits(paged, cols=0) == 0
    if paged:
        for kw in (dict(cache_rows=-1), dict(req=None), dict(ends=None), dict(table=None), dict(t_rows=-1),
                   dict(t_cols=-1), dict(ld_t=3), dict(block=0), dict(stride=-1), dict(req=ODD), dict(table=ODD)):
            assert logits(True, **kw) == EINVAL, kw
        assert logits(True, cache_rows=1 << 31) == EUNSUP


def rows(**kw):
    a = dict(q=P, rows=4, heads=16, dl=512, dr=64, ld_q=16 * 576, ld_head=576, cache=P, cache_rows=64, ld_cache=576,
             ids=P, k=32, ld_ids=32, counts=P, scale=0.1, out=P, lse=P, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.latent_attend_rows(*a.values(), None)


def paged(**kw):
    a = dict(q=P, rows=4, heads=16, dl=512, dr=64, ld_q=16 * 576, ld_head=576, cache=P, cache_rows=64, ld_cache=576,
             starts=P, ctx=P, reqs=2, tree=P, table=P, t_cols=4, ld_t=4, block=16, stride=16, max_len=64, scale=0.1,
             out=P, lse=P, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.latent_attend_paged(*a.values(), None)


@pytest.mark.parametrize("call", [rows, paged])
def test_latent_refusals(call):
    for kw in (dict(rows=-1), dict(heads=0), dict(dl=0), dict(dr=-1), dict(cache_rows=-1), dict(ld_cache=575),
               dict(ld_head=575), dict(ld_q=-8), dict(q=None), dict(out=None), dict(cache=None), dict(q=ODD),
               dict(cache=ODD), dict(out=ODD), dict(lse=ODD), dict(ld_q=9220), dict(ld_head=580), dict(ld_cache=580),
               dict(ws_bytes=64)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(dl=128), dict(dr=32), dict(heads=1025), dict(rows=1 << 28), dict(cache_rows=1 << 31)):
        assert call(**kw) == EUNSUP, kw
    assert call(rows=0) == 0


def test_latent_own_refusals():
    for kw in (dict(k=-1), dict(ld_ids=31), dict(ids=None), dict(ids=ODD), dict(counts=ODD)):
        assert rows(**kw) == EINVAL, kw
    for kw in (dict(reqs=-1), dict(max_len=-1), dict(t_cols=-1), dict(ld_t=3), dict(block=0), dict(stride=-1),
               dict(starts=None), dict(ctx=None), dict(table=None), dict(starts=ODD), dict(ctx=ODD), dict(tree=ODD)):
        assert paged(**kw) == EINVAL, kw
    assert paged(reqs=0) == 0


def test_latent_workspace_sizes():
    assert lib.latent_attend_rows_workspace_size(0, 16, 512, 64) == 0
    assert lib.latent_attend_rows_workspace_size(4, 16, 100, 64) == 0
    assert lib.latent_attend_paged_workspace_size(4, 0, 16, 512, 64) == 0
    assert lib.latent_attend_paged_workspace_size(4, 2, 0, 512, 64) == 0
    assert lib.latent_attend_rows_workspace_size(1 << 40, 16, 512, 64) == 0
    need = lib.latent_attend_rows_workspace_size(1, 16, 512, 2048)
    if need:
        assert rows(rows=1, k=2048, ld_ids=2048, ws=P, ws_bytes=need - 16) == EWS
        assert rows(rows=1, k=2048, ld_ids=2048, ws=ctypes.c_void_p(0x10004), ws_bytes=need) == EINVAL
    need = lib.latent_attend_paged_workspace_size(1, 1, 16, 512, 8192)
    if need:
        assert paged(rows=1, reqs=1, max_len=8192, ws=P, ws_bytes=need - 16) == EWS


def test_merge_refusals():
    def merge(**kw):
        a = dict(parts=P, dtype=1, lse=P, world=2, rows=4, heads=16, dim=512, out=P, odt=1, out_lse=P)
        a.update(kw)
        return lib.merge_attend_rank_major(*a.values(), None)

    for kw in (dict(dtype=2), dict(odt=2), dict(world=0), dict(world=65), dict(rows=-1), dict(heads=0), dict(dim=0),
               dict(dim=12), dict(parts=None), dict(lse=None), dict(out=None), dict(parts=ODD), dict(lse=ODD),
               dict(out=ODD), dict(out_lse=ODD)):
        assert merge(**kw) == EINVAL, kw
    assert merge(dim=2056) == EUNSUP and merge(rows=1 << 30) == EUNSUP
    assert merge(rows=0) == 0


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        rts.assign_slots(z(2, **i), z(2, **i), 4, z(2, 2, **i), z(4, **i), 16)
    with pytest.raises(ValueError):
        rts.indexer_logits(z(2, 8, 128, dtype=torch.bfloat16), z(4, 128, dtype=torch.bfloat16), z(2, 8))
    with pytest.raises(ValueError):
        rts.latent_attend_rows(z(2, 8, 576, dtype=torch.bfloat16), z(4, 576, dtype=torch.bfloat16), z(2, 3, **i), 0.1)
    with pytest.raises(ValueError):
        rts.latent_attend_paged(z(2, 8, 576, dtype=torch.bfloat16), z(4, 576, dtype=torch.bfloat16), z(3, **i),
                                z(2, **i), z(2, 1, **i), 2, 0.1)
    with pytest.raises(ValueError):
        rts.merge_attend_rank_major(z(2, 3, 8, 512), z(2, 3, 8))
