"""Host side of the operators from a prompt to a bounded cache (bsa_rope_*,
bsa_cache_weigh, bsa_cache_evict): sizes and argument checks, which return before
the library touches a device (the pointers are host addresses that are never
dereferenced), and pins of their oracles."""
import ctypes
import math

import numpy as np
import pytest

from block_sparse_attention_plan_gb300 import _cache as C
from block_sparse_attention_plan_gb300 import _prompt as P
from oracle import cache as OC
from oracle import prompt as OP

VP = ctypes.c_void_p


@pytest.fixture()
def lib(bsa):
    C._library()
    return P._library()


@pytest.fixture()
def buf():
    b = (ctypes.c_uint8 * 8192)()
    b.at = (ctypes.addressof(b) + 255) & ~255
    return b


def cache(buf, **kw):
    f = dict(k=buf.at, v=buf.at, k_scale=buf.at, v_scale=buf.at, block_table=buf.at, seq_lens=buf.at,
             page_refs=buf.at, control=buf.at, kind=0, num_pages=8, Hkv=2, page_size=64, d=128, scale_block=32,
             max_seqs=4, max_pages=6)
    f.update(kw)
    return C.CacheC(*(f[n] for n, _ in C.CacheC._fields_))


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("rot,base,scaling,factor,original", [
    (128, 10000.0, "none", 1.0, 0), (64, 500000.0, "linear", 4.0, 0), (32, 10000.0, "base", 8.0, 0),
    (128, 10000.0, "parts", 16.0, 4096), (16, 100.0, "parts", 1.0, 1)])
def test_steps_are_the_frequencies(lib, rot, base, scaling, factor, original):
    words, amp = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    assert lib.bsa_rope_steps(rot, base, P._SCALINGS[scaling], factor, original, words, ctypes.byref(amp)) == 0
    f, a = OP.frequencies(rot, base, scaling, factor, original)
    got = np.array([w / 2.0 ** 64 * 2 * math.pi for w in words[:rot // 2]])
    # doubles throughout: a few rounding steps of 2^-53, and pow's
    assert np.allclose(got, f, rtol=1e-14, atol=2.0 ** -60)
    assert amp.value == pytest.approx(a, rel=2.0 ** -23)
    assert all(w == 0 for w in words[rot // 2:])


@pytest.mark.parametrize("args,status", [
    ((0, 10000.0, 0, 1.0, 0.0), -1), ((24, 10000.0, 0, 1.0, 0.0), -1), ((144, 10000.0, 0, 1.0, 0.0), -1),
    ((64, 1.0, 0, 1.0, 0.0), -1), ((64, math.nan, 0, 1.0, 0.0), -1), ((64, math.inf, 0, 1.0, 0.0), -1),
    ((64, 1e4, 4, 1.0, 0.0), -2), ((64, 1e4, -1, 1.0, 0.0), -2), ((64, 1e4, 1, 0.5, 0.0), -1),
    ((64, 1e4, 2, math.nan, 0.0), -1), ((64, 1e4, 3, 2.0, 0.0), -1), ((64, 1e4, 3, math.inf, 4096.0), -1)])
def test_steps_refuse(lib, args, status):
    words, amp = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    assert lib.bsa_rope_steps(*args, words, ctypes.byref(amp)) == status


def test_rope_apply_refuses(lib, buf):
    def rope(**kw):
        f = dict(steps=buf.at, amplitude=1.0, rot=64, pairs=0)
        f.update(kw)
        return P.RopeC(*f.values())

    def call(r, q=None, o=None, Hq=4, Hk=0, dtype=0, pos=None, B=2, T=3, d=128, flags=0, k=None, ko=None):
        good = C.RowsC(buf.at, 512, 128, 1024)
        return lib.bsa_rope_apply(r, q or good, o or good, Hq, k, ko, Hk, dtype, pos, B, T, d, flags, None)

    good = C.RowsC(buf.at, 512, 128, 1024)
    odd = VP(buf.at + 2)
    cases = [(call(None), -1), (call(rope(steps=None)), -1), (call(rope(steps=buf.at + 4)), -1), (call(rope(rot=0)), -2),
             (call(rope(rot=24)), -2), (call(rope(rot=144)), -2), (call(rope(), d=96), -2), (call(rope(rot=128), d=64), -2),
             (call(rope(pairs=2)), -2), (call(rope(amplitude=math.nan)), -1), (call(rope(amplitude=math.inf)), -1),
             (call(rope(), dtype=2), -2), (call(rope(), B=0), -1), (call(rope(), T=0), -1), (call(rope(), Hq=0), -1),
             (call(rope(), Hk=-1), -1), (call(rope(), flags=2), -1), (call(rope(), pos=odd), -1),
             (call(rope(), Hk=2), -1),                                                # no k
             (call(rope(), Hk=2, k=good, ko=C.RowsC(buf.at, 0, 128, 256)), -1),       # rows written twice
             (call(rope(), o=C.RowsC(buf.at, 512, 0, 1024)), -1), (call(rope(), o=C.RowsC(buf.at, 512, 128, 0)), -1),
             (call(rope(), q=C.RowsC(buf.at + 8, 512, 128, 1024)), -1), (call(rope(), q=C.RowsC(buf.at, 512, 129, 1024)), -1),
             (call(rope(), q=C.RowsC(buf.at, -512, 128, 1024)), -1), (call(rope(), B=1 << 16, T=1 << 16), -2)]
    for i, (got, want) in enumerate(cases):
        assert got == want, i


def test_prompt_attention_refuses(lib, buf):
    good = lambda H: C.RowsC(buf.at, 0, 64, H * 64)
    size = lib.bsa_prompt_workspace_bytes(2, 10, 4, 2)

    def call(q=good(4), k=good(2), v=good(2), o=good(4), lse=VP(buf.at), dtype=0, off=VP(buf.at), n=2, T=10, Hq=4, Hkv=2, d=64, flags=0,
             scale=0.0, ws=VP(buf.at), nbytes=size):
        return lib.bsa_prompt_attention(q, k, v, o, lse, dtype, off, n, T, Hq, Hkv, d, flags, scale, ws, nbytes, None)

    odd = VP(buf.at + 2)
    cases = [(call(q=None), -1), (call(k=None), -1), (call(v=None), -1), (call(o=None), -1), (call(off=None), -1), (call(ws=None), -1),
             (call(off=odd), -1), (call(lse=odd), -1), (call(ws=VP(buf.at + 8)), -1), (call(nbytes=size - 1), -5), (call(nbytes=0), -5),
             (call(flags=2), -1), (call(scale=math.nan), -1), (call(scale=math.inf), -1), (call(dtype=2), -2), (call(d=96), -2),
             (call(n=0), -1), (call(T=0), -1), (call(Hq=0), -1), (call(Hkv=0), -1), (call(Hq=5), -1),
             (call(T=(1 << 30) + 1), -2), (call(Hq=65538), -2)]
    for rows in ("q", "k", "v", "o"):
        cases += [(call(**{rows: C.RowsC(buf.at + 8, 0, 64, 256)}), -1), (call(**{rows: C.RowsC(None, 0, 64, 256)}), -1),
                  (call(**{rows: C.RowsC(buf.at, 0, 64, 257)}), -1), (call(**{rows: C.RowsC(buf.at, 0, 68, 256)}), -1),
                  (call(**{rows: C.RowsC(buf.at, 0, 64, -256)}), -1), (call(**{rows: C.RowsC(buf.at, 0, 64, 0)}), -1),
                  (call(**{rows: C.RowsC(buf.at, 0, 0, 256)}), -1), (call(**{rows: C.RowsC(buf.at, 0, 64, 1 << 38)}), -1)]
    for i, (got, want) in enumerate(cases):
        assert got == want, i


def test_prompt_workspace_sizes(lib):
    size = lib.bsa_prompt_workspace_bytes
    assert 0 < size(1, 1, 1, 1) <= size(64, 4096, 32, 8) <= size(65, 4096, 32, 8) < size(65, 1 << 20, 32, 8)
    # an item for every 256 rows of a group of heads (tokens x heads that go together) and one more for each prompt
    for n, T, Hq, Hkv, gp in ((1, 100000, 8, 8, 1), (7, 100000, 32, 1, 16), (3, 50000, 28, 4, 1), (3, 50000, 24, 4, 2)):
        assert size(n, T, Hq, Hkv) >= 16 * (T * gp // 256 + n) + 4 * (n + 1) + 64
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 3, 2), (1, (1 << 30) + 1, 1, 1), (1, 1, 65538, 1)):
        assert size(*bad) == 0


def test_rotation_oracle():
    x = np.random.default_rng(0).standard_normal((5, 3, 7, 32))
    f, _ = OP.frequencies(16)
    pos = np.arange(7) * 1000
    for pairs in ("half", "neighbours"):
        y = OP.rotate(x, pos, f, 1.5, pairs)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(np.square(y[..., :16]).sum(-1), 2.25 * np.square(x[..., :16]).sum(-1))  # amp times a rotation
        assert np.allclose(OP.rotate(y, pos, f, 1 / 1.5, pairs, inverse=True), x)
        # a product depends on the distance of two positions alone
        a, b = x[0, 0, :1], x[1, 0, :1]
        s = [OP.rotate(a, [p], f, 1.0, pairs)[0, :16] @ OP.rotate(b, [p - 5], f, 1.0, pairs)[0, :16] for p in (5, 900)]
        assert s[0] == pytest.approx(s[1], rel=1e-10)
    y = OP.rotate(np.eye(16)[:1], [1.0], f, 1.0, "half")  # element 0 turns towards its partner by one radian
    assert y[0, 0] == pytest.approx(math.cos(1)) and y[0, 8] == pytest.approx(math.sin(1))


# ------------------------------------------------------------------ weights and eviction

def test_weigh_refuses(lib, buf):
    c, r, p = cache(buf), C.RowsC(buf.at, 0, 128, 128), VP(buf.at)
    call = lambda c=c, q=r, lse=p, dtype=0, seqs=None, mask=None, NKB=0, bk=0, B=1, Hq=4, nq=1, flags=0, scale=0.0, fresh=0, w=p, tokens=384: \
        lib.bsa_cache_weigh(c, q, lse, dtype, seqs, mask, NKB, bk, B, Hq, nq, flags, scale, fresh, w, tokens, None)
    odd = VP(buf.at + 2)
    for got, want in [(call(c=None), -1), (call(c=cache(buf, d=96)), -2), (call(c=cache(buf, k=None)), -1), (call(lse=None), -1),
                      (call(lse=odd), -1), (call(w=None), -1), (call(w=odd), -1), (call(tokens=0), -1), (call(fresh=-1), -1),
                      (call(dtype=2), -2), (call(seqs=odd), -1), (call(flags=2), -1), (call(scale=math.nan), -1),
                      (call(scale=math.inf), -1), (call(B=0), -1), (call(B=5), -1), (call(Hq=3), -1), (call(nq=0), -1),
                      (call(mask=p, NKB=4, bk=48), -2), (call(mask=p, NKB=0, bk=64), -1),
                      (call(q=C.RowsC(buf.at + 8, 0, 128, 128)), -1), (call(q=C.RowsC(buf.at, 4, 128, 128)), -1)]:
        assert got == want


def test_evict_refuses(lib, buf):
    c, p = cache(buf), VP(buf.at)
    call = lambda c=c, w=p, tokens=384, seqs=None, keep=p, sink=0, recent=0, kept=p, most=64, n=2, ws=p, nbytes=256: \
        lib.bsa_cache_evict(c, w, tokens, seqs, keep, sink, recent, kept, most, n, ws, nbytes, None)
    odd = VP(buf.at + 2)
    for got, want in [(call(c=None), -1), (call(c=cache(buf, page_size=48)), -2), (call(w=None), -1), (call(w=odd), -1),
                      (call(tokens=0), -1), (call(seqs=odd), -1), (call(keep=None), -1), (call(keep=odd), -1), (call(sink=-1), -1),
                      (call(recent=-1), -1), (call(kept=None), -1), (call(kept=odd), -1), (call(most=0), -1), (call(n=0), -1),
                      (call(n=5), -1), (call(n=4097, seqs=p), -2), (call(ws=None), -1), (call(ws=odd), -1), (call(nbytes=255), -5)]:
        assert got == want
    assert lib.bsa_cache_evict_workspace_bytes(1) >= 4 and lib.bsa_cache_evict_workspace_bytes(65) > lib.bsa_cache_evict_workspace_bytes(1)
    assert lib.bsa_cache_evict_workspace_bytes(0) == 0 and lib.bsa_cache_evict_workspace_bytes(4097) == 0


def test_weights_of_the_oracle_sum_to_the_rows():
    """Over all keys that a row sees, its weights sum to 1 where LSE is its own."""
    m = OC.CacheModel(6, 2, 16, 64, 2, 3, seed=3)
    m.resize([37, 20])
    rng = np.random.default_rng(0)
    m.append(rng.standard_normal((2, 2, 37, 64)), rng.standard_normal((2, 2, 37, 64)), counts=[37, 20])
    q = rng.standard_normal((2, 4, 3, 64))
    w = np.full((2, 2, 48), 7.0)
    lse = np.empty((2, 4, 3))
    for b, n in enumerate((37, 20)):
        k, v = m.values(b)
        see = np.array([[[j <= n - 3 + i for j in range(n)] for i in range(3)]] * 4)
        lse[b] = OC.attention(q[b], k, v, see)[1]
    m.weigh(w, q, lse, keep=lambda b, h, i, j: j <= m.lens[b] - 3 + i, fresh=1 << 30)
    assert np.allclose(w[0, :, :37].sum(-1), 6) and np.allclose(w[1, :, :20].sum(-1), 6)
    assert (w[0, :, 37:] == 7).all() and (w[1, :, 20:] == 7).all()


def test_eviction_of_the_oracle_by_hand():
    m = OC.CacheModel(4, 1, 16, 64, 1, 4, "int8", 16, seed=0)
    m.resize([40])
    m.append(np.arange(40.0).reshape(1, 1, 40, 1).repeat(64, 3), np.ones((1, 1, 40, 64)))
    w = np.zeros((1, 1, 64))
    w[0, 0, [5, 9, 30]] = 3.0, 1.0, 2.0
    w[0, 0, 20] = math.nan
    kept = m.evict(w, [8], sink=2, recent=2)
    # sinks 0, 1; 5, 30 and 9 by weight, then 2, the first of those without; the last two
    assert kept == [[[0, 1, 2, 5, 9, 30, 38, 39]]]
    assert m.lens[0] == 8 and m.refs.sum() == 1 and (m.table[0, 1:] == -1).all()
    assert np.array_equal(m.values(0)[0][0, :, 0], [0, 1, 2, 5, 9, 30, 38, 39])
    assert list(w[0, 0, :8]) == [0, 0, 0, 3, 1, 2, 0, 0]
    assert m.evict(w, [8]) == [[list(range(8))]]
