"""kv_attend_paged: windows and lengths at the ends of their range, split and whole."""

import pytest

from gpu_common import say
from test_gpu_kv_attend import E4M3, check, plan, rts, setup  # noqa: F401 (rts: the fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("ends,window", [
    ([70, 64, 63, 65], 16), ([79, 80, 81, 1 << 20], 16), ([2 ** 31 - 1] * 4, 16), ([2 ** 31 - 1] * 4, 2 ** 31 - 64),
    ([70, 1, 0, -5], 1), ([65, 66, 128, 129], 65), ([70, 71, 72, 73], 1 << 40)])
def test_window_of_a_row_that_ends_past_its_table(rts, dtype, ends, window):  # noqa: F811
    """The window counts back from the row's end, wherever the table's is."""
    say("window past the table", dtype, ends, window)
    q, k, v, req, _, table = setup(17, [64] * 4, 4, 2, 64, 16, dtype=dtype)
    for ws in ("auto", None):
        check(rts, q, k, v, req, ends, table, 16, 0.125, window=window, workspace=ws)


@pytest.mark.parametrize("past", [1, 700, 4999, 5000, 6000])
def test_window_past_the_table_split(rts, past):  # noqa: F811
    say("split window past the table", past)
    window = 5000
    assert plan(rts, 3, 2, 1, 64, 1 << 20, window)[0] > 1
    q, k, v, req, _, table = setup(18, [6000, 6000, 6000], 2, 1, 64, 16)
    for ws in ("auto", None):
        check(rts, q, k, v, req, [6000 + past, 6000, 5999], table, 16, 0.125, window=window, max_len=1 << 20, workspace=ws)
