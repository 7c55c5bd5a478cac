"""Host side of the 8-bit cache's C entry points: sizes and argument checks,
which return before the library touches a device (the pointers are host
addresses that are never dereferenced)."""
import ctypes

import pytest

from block_sparse_attention_plan_gb300 import _cache as C

VP = ctypes.c_void_p


@pytest.fixture()
def lib(bsa):
    return C._library()


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


def test_control_bytes(lib):
    assert lib.bsa_cache_control_bytes(8) == 4 * (16 + 3 * 8)
    assert lib.bsa_cache_control_bytes(0) == 0
    assert lib.bsa_cache_control_bytes(1 << 30) > 1 << 33


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), -1), (dict(control=None), -1), (dict(kind=2), -2), (dict(d=96), -2), (dict(page_size=48), -2),
    (dict(page_size=8, scale_block=8), -2), (dict(page_size=512), -2), (dict(scale_block=128), -2),
    (dict(scale_block=8), -2), (dict(num_pages=0), -1), (dict(Hkv=0), -1), (dict(max_seqs=0), -1),
    (dict(max_pages=0), -1), (dict(num_pages=1 << 30, Hkv=64), -2), (dict(max_pages=1 << 28), -2)])
def test_cache_struct_is_checked_by_every_call(lib, buf, kw, status):
    c = cache(buf, **kw)
    p = VP(buf.at)
    r = C.RowsC(buf.at, 0, 128, 128)
    good = cache(buf)
    for got in (lib.bsa_cache_init(c, None), lib.bsa_cache_status(c, None, None), lib.bsa_cache_resize(c, p, p, 2, None),
                lib.bsa_cache_fork(c, p, p, 2, None), lib.bsa_cache_compact(c, None),
                lib.bsa_cache_copy_pages(c, good, p, p, 1, None), lib.bsa_cache_copy_pages(good, c, p, p, 1, None),
                lib.bsa_cache_append(c, r, r, 0, None, None, None, 1, 1, None),
                lib.bsa_cache_attention(c, r, r, p, 0, None, None, 0, 0, 1, 2, 1, 0, 0.0, p, 1 << 30, None),
                lib.bsa_cache_forward(p, c, None, p, 0, p, p, 0.0, p, 1 << 30, None)):
        assert got == status, kw
    assert lib.bsa_cache_attention_workspace_bytes(c, 1, 2, 1, 0, 0) == 0


def test_null_and_misaligned_structs(lib, buf):
    assert lib.bsa_cache_init(None, None) == -1
    for field in ("k", "v"):
        assert lib.bsa_cache_init(cache(buf, **{field: buf.at + 8}), None) == -1
    for field in ("k_scale", "block_table", "seq_lens", "page_refs", "control"):
        assert lib.bsa_cache_init(cache(buf, **{field: buf.at + 2}), None) == -1


def test_call_arguments(lib, buf):
    c, p = cache(buf), VP(buf.at)
    r = C.RowsC(buf.at, 256, 128, 128)
    assert lib.bsa_cache_resize(c, p, p, 0, None) == -1
    assert lib.bsa_cache_resize(c, None, p, 5, None) == -1      # 5 of 4 sequences
    assert lib.bsa_cache_resize(c, p, p, 4097, None) == -2
    assert lib.bsa_cache_resize(c, VP(buf.at + 2), p, 1, None) == -1
    assert lib.bsa_cache_fork(c, None, p, 1, None) == -1
    assert lib.bsa_cache_fork(c, p, p, 4097, None) == -2
    assert lib.bsa_cache_copy_pages(c, c, p, p, 9, None) == -1  # 9 of 8 pages
    for other in (dict(kind=1), dict(Hkv=1), dict(page_size=32), dict(d=64), dict(scale_block=16), dict(num_pages=9)):
        assert lib.bsa_cache_copy_pages(c, cache(buf, **other), p, p, 1, None) == -1, other
    app = lambda k=r, v=r, dt=0, n=1, T=1, seqs=None: lib.bsa_cache_append(c, k, v, dt, seqs, None, None, n, T, None)
    assert app(n=0) == -1 and app(T=0) == -1 and app(n=5) == -1 and app(T=385) == -1 and app(dt=2) == -2
    for bad in (C.RowsC(None, 256, 128, 128), C.RowsC(buf.at + 8, 256, 128, 128), C.RowsC(buf.at, 4, 128, 128),
                C.RowsC(buf.at, 256, -128, 128), C.RowsC(buf.at, 256, 128, 12)):
        assert app(k=bad) == -1 and app(v=bad) == -1

    def att(q=r, o=r, lse=p, dt=0, mask=None, NKB=0, bk=0, B=1, Hq=2, nq=1, flags=0, scale=0.0, ws=p, n=1 << 30):
        return lib.bsa_cache_attention(c, q, o, lse, dt, None, mask, NKB, bk, B, Hq, nq, flags, scale, ws, n, None)

    for n, bad in ((dict(B=2), C.RowsC(buf.at, 0, 128, 128)), (dict(Hq=4), C.RowsC(buf.at, 512, 0, 128)),
                   (dict(nq=2), C.RowsC(buf.at, 512, 256, 0))):
        assert att(o=bad, **n) == -1, n                         # rows of o that are one
    assert att(B=0) == -1 and att(Hq=3) == -1 and att(nq=0) == -1 and att(B=5) == -1
    assert att(flags=2) == -1 and att(dt=2) == -2 and att(scale=float("nan")) == -1 and att(scale=float("inf")) == -1
    assert att(mask=p, NKB=4, bk=48) == -2 and att(mask=p, NKB=0, bk=64) == -1
    assert att(ws=None) == -1 and att(ws=VP(buf.at + 8)) == -1 and att(lse=VP(buf.at + 2)) == -1
    need = lib.bsa_cache_attention_workspace_bytes(c, 1, 2, 1, 0, 0)
    assert need > 0 and att(n=need - 1) == -5
    masked = lib.bsa_cache_attention_workspace_bytes(c, 1, 2, 1, 4, 64)
    assert masked > need and att(mask=p, NKB=4, bk=64, n=masked - 1) == -5


def test_forward_arguments(lib, buf):
    c, p = cache(buf), VP(buf.at)
    assert lib.bsa_cache_forward(None, c, None, p, 0, p, p, 0.0, p, 1 << 30, None) == -1
    assert lib.bsa_cache_forward(p, c, None, p, 0, p, p, 0.0, p, 1 << 30, None) == -7  # no plan of this library
    assert lib.bsa_cache_forward_workspace_bytes(None, c) == 0
