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
