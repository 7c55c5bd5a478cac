"""Pins of the cache oracle's rule for a block's scale: what was stored counts,
what the page's last holder left does not."""
import numpy as np
import pytest

from oracle import cache as OC


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("left", [2.0 ** 20, np.nan, np.inf, 0.0])
def test_pieces_give_the_scale_of_one_call(kind, left):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 2, 100, 8))
    models = []
    for pieces in ([(0, 100)], [(0, 40), (40, 60)], [(90, 10), (20, 70), (0, 20)], [(i, 1) for i in range(100)]):
        m = OC.CacheModel(4, 2, 32, 8, 1, 4, kind, 16, seed=2)
        for s in m.scales:
            s[:] = left
        assert m.resize([100]) == 0
        for at, n in pieces:
            m.append(x[:, :, at:at + n], -x[:, :, at:at + n], start=[at])
        models.append(m)
    for m in models[1:]:
        for a, b in zip(m.scales, models[0].scales):
            held = np.arange(a.shape[0] * a.shape[2]).reshape(a.shape[0], 1, a.shape[2]) < 7  # ceil(100 / 16) blocks
            assert np.array_equal(np.where(held, a, 0), np.where(held, b, 0))


def test_a_step_of_one_token_writes_no_scales():
    m = OC.CacheModel(6, 1, 16, 8, 2, 3, "int8", 16, seed=2)
    assert m.resize([16, 5]) == 0
    for s in m.scales:
        s[:] = 3.0
    assert m.resize([17, 6]) == 0
    assert all((s == 3.0).all() for s in m.scales)
    assert m.resize([18, 17]) == 0  # (the second enters a block with one token, but grows by eleven)
    assert all((s == 3.0).sum() == s.size - 1 for s in m.scales)
