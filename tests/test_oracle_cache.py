"""Pins of the cache oracle: the code tables, rounding against torch's types,
attention against torch's fp64 softmax, the page bookkeeping's invariants."""
import numpy as np
import pytest
import torch

from oracle import cache as OC


def test_e4m3_table_matches_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(OC.decode(codes, "e4m3"), t, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 100, rng.standard_normal(5000) * 0.01, [448, 463, 500, 0.0],
                        (OC.e4m3_values()[:126] + OC.e4m3_values()[1:127]) / 2])   # every tie
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OC.encode(x, "e4m3"), want)
    y = np.concatenate([x, np.arange(-130, 130) + 0.5])
    assert np.array_equal(OC.encode(y, "int8").view(np.int8), np.clip(np.rint(y), -127, 127).astype(np.int8))


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_scale_is_the_smallest_power_of_two(kind):
    for a in [0.0, 1e-40, 1.0, 3.5, 7.0, 7.9375, 448.0, 448.5, 127.0, 128.0, 3e38]:
        s = OC.scale_for(a, kind)
        assert np.log2(s) == round(np.log2(s)) and a <= OC.TOP[kind] * s
        assert s == OC.MIN_SCALE or a > OC.TOP[kind] * s / 2


def test_attention_matches_torch_softmax():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(h, n, 16, generator=g, dtype=torch.float64) for h, n in ((4, 3), (2, 50), (2, 50)))
    keep = torch.rand(4, 3, 50, generator=g) < 0.5
    keep[1, 2] = False
    O, lse, _, _ = OC.attention(q.numpy(), k.numpy(), v.numpy(), keep.numpy())
    kk, vv = k.repeat_interleave(2, 0), v.repeat_interleave(2, 0)
    s = (q @ kk.transpose(1, 2) / 4.0).masked_fill(~keep, float("-inf"))
    w = torch.softmax(s, -1).nan_to_num(0.0)
    assert np.allclose(O, (w @ vv).numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-12)
    assert np.isneginf(lse[1, 2]) and not O[1, 2].any()


def test_page_bookkeeping_invariants():
    rng = np.random.default_rng(5)
    m = OC.CacheModel(40, 1, 16, 8, 8, 6)
    for _ in range(300):
        op = rng.integers(4)
        if op == 0:
            seqs = rng.choice(8, 3, replace=False)
            before = (m.table.copy(), m.lens.copy(), m.refs.copy())
            if m.resize(rng.integers(0, 97, 3), seqs):
                assert all(np.array_equal(a, b) for a, b in zip(before, (m.table, m.lens, m.refs)))
        elif op == 1:
            m.resize([0], [rng.integers(8)])
        elif op == 2:
            empty = np.nonzero(m.lens == 0)[0]
            full = np.nonzero(m.lens)[0]
            if len(empty) and len(full):
                m.fork([full[0]], [empty[-1]])
        else:
            L = m.compact()
            assert (m.refs[:L] > 0).all() and (m.refs[L:] == 0).all()
        held = [m.table[s, j] for s in range(8) for j in range(m._pages(m.lens[s]))]
        assert np.array_equal(np.bincount(np.array(held, dtype=int), minlength=40), m.refs)
        for s in range(8):  # no page past the length; a partly filled last page of a grown sequence is its own
            assert (m.table[s, m._pages(m.lens[s]):] == -1).all()


def test_append_leaves_shared_pages_alone():
    m = OC.CacheModel(8, 1, 16, 8, 4, 3, seed=1)
    assert m.resize([20], [0]) == 0
    x = np.random.default_rng(2).standard_normal((1, 1, 20, 8))
    m.append(x, x, [0])
    m.fork([0], [1])
    before = [a.copy() for a in m.codes + m.scales]
    m.append(x[:, :, :5], x[:, :, :5], [1])
    assert all(np.array_equal(a, b) for a, b in zip(before, m.codes + m.scales))
    assert m.resize([22], [1]) == 0
    m.append(x[:, :, :6], x[:, :, :6], [1])  # tokens 16 .. 21, in a page of its own
    k0, k1 = m.values(0)[0], m.values(1)[0]
    assert np.array_equal(k0[:, :16], k1[:, :16]) and not np.array_equal(k0[:, 16:20], k1[:, 16:20])
