"""Refusals of the serving-path entry points that other files do not hold (host only)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import row_top_select_amd as rts  # noqa: E402

i64 = ctypes.c_int64
lib = rts.raw_library()


def test_indexer_logits_plan():
    f, p = lib.indexer_logits_plan, (i64 * 4)()
    for bad in ((0, i64(4), 8, 128, i64(64), i64(-1), p), (1, i64(0), 8, 128, i64(64), i64(-1), p),
                (1, i64(4), 0, 128, i64(64), i64(-1), p), (1, i64(4), 8, 128, i64(0), i64(-1), p),
                (1, i64(4), 8, 128, i64(64), i64(-2), p), (1, i64(4), 8, 128, i64(64), i64(-1), None)):
        assert f(*bad) == -1, bad
    for bad in ((1, i64(4), 129, 128, i64(64), i64(-1), p), (1, i64(4), 8, 96, i64(64), i64(-1), p),
                (1, i64(4), 8, 128, i64(1 << 31), i64(-1), p)):
        assert f(*bad) == -2, bad
    assert f(1, i64(3), 8, 128, i64(64), i64(-1), p) == 0
    tokens, steps, step, stages = p
    assert 1 <= tokens <= 3 and steps >= 1 and step in (256, 512) and stages in (1, 2)


def test_latent_plans():
    rows, paged, p = lib.latent_attend_rows_plan, lib.latent_attend_paged_plan, (ctypes.c_int32 * 2)()
    for bad in ((i64(0), 16, 512, 64, 1, p), (i64(4), 0, 512, 64, 1, p), (i64(4), 16, 512, -1, 1, p),
                (i64(4), 16, 512, 64, 1, None)):
        assert rows(*bad) == -1, bad
    for bad in ((i64(0), i64(2), 16, 512, i64(64), 1, p), (i64(4), i64(0), 16, 512, i64(64), 1, p),
                (i64(4), i64(2), 0, 512, i64(64), 1, p), (i64(4), i64(2), 16, 512, i64(-1), 1, p),
                (i64(4), i64(2), 16, 512, i64(64), 1, None)):
        assert paged(*bad) == -1, bad
    assert rows(i64(4), 1025, 512, 64, 1, p) == -2 and rows(i64(1 << 31), 16, 512, 64, 1, p) == -2
    assert rows(i64(4), 16, 128, 64, 1, p) == -2 and paged(i64(4), i64(2), 16, 128, i64(64), 1, p) == -2
    assert paged(i64(1 << 31), i64(2), 16, 512, i64(64), 1, p) == -2
    for f, a in ((rows, (i64(2), 16, 512, 2048)), (paged, (i64(2), i64(2), 16, 512, i64(4096)))):
        assert f(*a, 0, p) == 0 and p[0] in (1, 2, 4) and p[1] == 1
        assert f(*a, 1, p) == 0 and p[0] in (1, 2, 4) and p[1] > 1


def test_inputs_that_require_gradients_are_refused():
    """The operators have no backward pass: a result without a graph would lose the gradients silently."""
    z = torch.zeros
    i = dict(dtype=torch.int32)
    b = dict(dtype=torch.bfloat16)
    q_i, keys, w, ks = z(2, 8, 128, **b), z(4, 128, **b), z(2, 8), z(4)
    q, cache = z(2, 8, 576, **b), z(4, 576, **b)
    parts, lse = z(2, 3, 8, 512), z(2, 3, 8)
    table = z(2, 1, **i)
    calls = [(lambda: rts.indexer_logits(q_i, keys, w, key_scales=ks), (q_i, keys, w, ks)),
             (lambda: rts.indexer_logits_paged(q_i, keys, w, z(2, **i), z(2, **i), table, 2, 2, key_scales=ks),
              (q_i, keys, w, ks)),
             (lambda: rts.latent_attend_rows(q, cache, z(2, 3, **i), 0.1), (q, cache)),
             (lambda: rts.latent_attend_paged(q, cache, z(3, **i), z(2, **i), table, 2, 0.1), (q, cache)),
             (lambda: rts.merge_attend_rank_major(parts, lse), (parts, lse))]
    for call, inputs in calls:
        for t in inputs:
            t.requires_grad_(True)
            with pytest.raises(ValueError, match="backward"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):  # as far as this goes without a GPU
                call()
            t.requires_grad_(False)


def test_scales_that_are_not_numbers_are_refused():
    p = ctypes.c_void_p(0x10000)  # never dereferenced
    for scale in (float("nan"), float("inf"), float("-inf"), 1.8e38, -3e38):
        assert lib.latent_attend_rows(p, 4, 16, 512, 64, 16 * 576, 576, p, 64, 576, p, 32, 32, p, scale, p, p, None, 0,
                                      None) == -1, scale
        assert lib.latent_attend_paged(p, 4, 16, 512, 64, 16 * 576, 576, p, 64, 576, p, p, 2, None, p, 4, 4, 16, 16, 64,
                                       scale, p, p, None, 0, None) == -1, scale
