"""What the binding of the beam step's operators hands to the library (no kernel runs in these tests)."""

import pytest

torch = pytest.importorskip("torch")

import row_top_select_amd as rts  # noqa: E402


@pytest.mark.parametrize("many", [lambda x: list(x), lambda x: tuple(x), lambda x: (t for t in x), lambda x: map(lambda t: t, x),
                                  lambda x: dict(enumerate(x)).values()], ids=["list", "tuple", "generator", "map", "view"])
def test_copy_blocks_takes_caches_of_any_iterable(monkeypatch, many):
    got = []
    monkeypatch.setattr(rts, "_gpu", lambda t, name: t.device)
    monkeypatch.setattr(rts, "_launch", lambda fn, where, device, stream, caches, n, *rest: got.append(
        [(c.data, c.rows, c.row_bytes, c.ld_bytes) for c in caches][:n]))
    caches = [torch.zeros(64, 3 + i % 2) for i in range(70)]  # more than one launch takes
    rts.copy_blocks(many(caches), torch.zeros(1, 2, dtype=torch.int32), 16)
    assert [len(x) for x in got] == [64, 6]
    assert sum(got, []) == [(t.data_ptr(), 64, t.shape[1] * 4, t.shape[1] * 4) for t in caches]


def test_copy_blocks_checks_every_cache_of_a_generator(monkeypatch):
    monkeypatch.setattr(rts, "_gpu", lambda t, name: t.device)
    monkeypatch.setattr(rts, "_launch", lambda *a: pytest.fail("launched"))
    pairs = torch.zeros(1, 2, dtype=torch.int32)
    good, other = torch.zeros(64, 3), torch.zeros(64, 3, device="meta")
    trained, rows = torch.zeros(64, 3, requires_grad=True), torch.zeros(64, 6)[:, ::2]
    for bad in (other, trained, rows):
        with pytest.raises(ValueError):
            rts.copy_blocks((t for t in (good, bad)), pairs, 16)


@pytest.mark.gpu
def test_copy_blocks_of_a_generator_copies():
    caches = [torch.arange(64 * 3, dtype=torch.float32, device="cuda").view(64, 3) + i for i in range(3)]
    want = [t.clone() for t in caches]
    for t in want:
        t[48:64] = t[16:32]
    rts.copy_blocks((t for t in caches), torch.tensor([[1, 3], [-1, -1]], dtype=torch.int32, device="cuda"), 16)
    assert all(torch.equal(a, b) for a, b in zip(caches, want))
