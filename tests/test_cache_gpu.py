"""GPU tests of the 8-bit paged cache (bsa_cache_*): every array of the page
operations and of appending bit for bit against the oracle's model, attention
and the forward over the cache against fp64 with bounds from the arithmetic."""
import numpy as np
import pytest
import torch

from oracle import cache as OC

pytestmark = pytest.mark.gpu

KINDS = ["e4m3", "int8"]


def upload(bsa, m, device="cuda"):
    """A Cache with the model's state."""
    dt = torch.float8_e4m3fn if m.kind == "e4m3" else torch.int8
    t = lambda a: torch.from_numpy(a.copy()).to(device)
    return bsa.Cache(*(t(x).view(dt) for x in m.codes), *(t(x) for x in m.scales), t(m.table), t(m.lens), t(m.refs))


def assert_state(c, m, what=""):
    for name, got, want in (("table", c.block_table, m.table), ("lens", c.lens, m.lens), ("refs", c.refs, m.refs)):
        assert np.array_equal(got.cpu().numpy(), want), (what, name)
    for name, got, want in (("k", c.k, m.codes[0]), ("v", c.v, m.codes[1])):
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want), (what, name)
    for name, got, want in (("k_scale", c.k_scale, m.scales[0]), ("v_scale", c.v_scale, m.scales[1])):
        assert np.array_equal(got.cpu().numpy(), want), (what, name)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen).to(dtype)


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("kind,page,sb,d", [("e4m3", 16, 16, 64), ("int8", 64, 32, 128)])
def test_page_operations_follow_the_model(bsa, kind, page, sb, d):
    rng = np.random.default_rng(11)
    m = OC.CacheModel(50, 2, page, d, 10, 7, kind, sb, seed=2)
    c = upload(bsa, m)
    for step in range(60):
        op = rng.integers(5)
        if op <= 1:
            n = int(rng.integers(1, 6))
            seqs = rng.choice(10, n, replace=False).astype(np.int32)
            lens = rng.integers(0, 7 * page + 1, n).astype(np.int32)
            bsa.cache_resize(c, torch.from_numpy(lens).cuda(), torch.from_numpy(seqs).cuda())
            missing = m.resize(lens, seqs)
            st, det = bsa.cache_status(c)
            assert (st, det) == ((-5, missing) if missing else (0, 0)), step
        elif op == 2:
            s = int(rng.integers(10))
            bsa.cache_free(c, i32(s, -1))
            m.resize([0], [s])
        elif op == 3:
            empty, full = np.nonzero(m.lens == 0)[0], np.nonzero(m.lens)[0]
            if len(empty) >= 2 and len(full):
                src = [int(full[0]), int(full[-1]), -1]
                dst = [int(empty[0]), int(empty[1]), int(empty[0])]
                bsa.cache_fork(c, i32(*src), i32(*dst))
                m.fork(src[:2], dst[:2])
        else:
            bsa.cache_compact(c)
            m.compact()
        assert_state(c, m, f"step {step} op {op}")
    assert bsa.cache_status(c) == (0, 0)


def test_copy_on_write_keeps_the_page_for_the_last(bsa):
    # Four sequences share a partly filled page and all grow in one call: three
    # take pages of their own, in order; the last keeps it.
    m = OC.CacheModel(12, 1, 16, 64, 4, 3, seed=4)
    c = upload(bsa, m)
    for f in (lambda x, *a: bsa.cache_resize(c, i32(*x), i32(*a)), lambda x, *a: m.resize(x, a)):
        f([20], 0)
    bsa.cache_fork(c, i32(0, 0, 0), i32(1, 2, 3))
    m.fork([0, 0, 0], [1, 2, 3])
    bsa.cache_resize(c, i32(21, 33, 21, 22), i32(2, 0, 3, 1))
    m.resize([21, 33, 21, 22], [2, 0, 3, 1])
    assert_state(c, m)
    assert m.table[1, 1] == 1 and len({m.table[s, 1] for s in range(4)}) == 4
    # A page that shrinking leaves partly filled is shared too.
    bsa.cache_resize(c, i32(5, 9), i32(0, 1))
    m.resize([5, 9], [0, 1])
    bsa.cache_resize(c, i32(6), i32(0))
    m.resize([6], [0])
    assert_state(c, m)


def test_resize_of_many_sequences_over_a_large_pool(bsa):
    m = OC.CacheModel(70000, 1, 16, 64, 3000, 30, seed=1)
    rng = np.random.default_rng(8)
    c = upload(bsa, m)
    for _ in range(3):
        lens = rng.integers(0, 25 * 16, 2900).astype(np.int32)
        bsa.cache_resize(c, torch.from_numpy(lens).cuda())
        assert m.resize(lens) == 0
        assert_state(c, m)
    bsa.cache_compact(c)
    m.compact()
    assert_state(c, m)


def test_copy_pages_between_caches(bsa):
    a, b = OC.CacheModel(9, 3, 32, 64, 2, 2, seed=1), OC.CacheModel(20, 3, 32, 64, 1, 1, seed=2)
    ca, cb = upload(bsa, a), upload(bsa, b)
    bsa.cache_copy_pages(cb, ca, i32(19, 0, 7), i32(8, 3, 3))
    for x, y in zip(a.codes + a.scales, b.codes + b.scales):
        y[[19, 0, 7]] = x[[8, 3, 3]]
    assert_state(cb, b)
    assert bsa.cache_status(cb) == (0, 0)
    # Within one cache: named twice, also a source, out of range.
    bsa.cache_copy_pages(cb, cb, i32(1, 2, 1, 5, 20, 6), i32(10, 11, 12, 13, 14, 5))
    for y in b.codes + b.scales:
        y[[1, 2]] = y[[10, 11]]
        y[6] = y[5]
    assert_state(cb, b)
    assert bsa.cache_status(cb)[0] == -1 and bsa.cache_status(cb) == (0, 0)


def test_bad_items_are_skipped_and_reported(bsa):
    m = OC.CacheModel(12, 1, 16, 64, 4, 3, seed=4)
    c = upload(bsa, m)
    cases = [((20, 5), (0, 0), 1), ((20, 5), (0, 4), 1), ((20, 49), (0, 1), 1), ((20, -1), (0, 1), 1), ((9, 9), (-2, 1), 0)]
    for lens, seqs, at in cases:
        bsa.cache_resize(c, i32(*lens), i32(*seqs))
        good = [i for i in range(2) if i != at]
        m.resize([lens[i] for i in good], [seqs[i] for i in good])
        assert bsa.cache_status(c) == (-1, at), (lens, seqs)
        assert_state(c, m)
    for src, dst in (((0,), (1,)), ((0, 0), (2, 2)), ((0, 2), (2, 3)), ((0,), (9,)), ((7,), (2,))):
        before = m.lens.copy()
        bsa.cache_fork(c, i32(*src), i32(*dst))
        assert bsa.cache_status(c)[0] == -1, (src, dst)
        if (src, dst) == ((0, 0), (2, 2)):
            m.fork([0], [2])
            assert_state(c, m)
            bsa.cache_free(c, i32(2))
            m.resize([0], [2])
        elif (src, dst) == ((0, 2), (2, 3)):   # 2 is a source: only the (empty) second pair happens
            m.fork([2], [3])
        assert_state(c, m)
    # Too few pages: nothing changes, not even the releases.
    bsa.cache_resize(c, i32(0, 48, 48, 48), i32(1, 0, 2, 3))
    assert m.resize([0, 48, 48, 48], [1, 0, 2, 3]) == 0
    bsa.cache_resize(c, i32(16, 48), i32(0, 1))
    assert m.resize([16, 48], [0, 1]) == 0
    assert_state(c, m)
    bsa.cache_resize(c, i32(48, 8), i32(0, 1))
    assert m.resize([48, 8], [0, 1]) == 0
    assert_state(c, m)


# ----------------------------------------------------------------- append

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page,sb,d,heads,dtype", [(64, 64, 128, 2, torch.bfloat16), (16, 16, 64, 3, torch.float16),
                                                   (256, 128, 128, 1, torch.bfloat16), (128, 32, 64, 2, torch.bfloat16),
                                                   (256, 256, 128, 1, torch.float16)])
def test_append_follows_the_model(bsa, kind, page, sb, d, heads, dtype):
    g = torch.Generator().manual_seed(page + sb)
    m = OC.CacheModel(12, heads, page, d, 4, 4, kind, sb, seed=3)
    m.resize([page + 5, 3, 2 * page, 1])
    c = upload(bsa, m)
    steps = [  # T, counts, growth of each sequence's scale
        (page + 5, (page + 5, 3, 40, 1), 1.0), (1, (1, 1, 1, 0), 0.1), (1, (1, 1, 1, 1), 30.0), (7, (5, 7, 0, 2), 1e4),
        (page // 2 + 3, (1, page // 2 + 3, 0, 9), 1e-3)]
    for T, counts, amp in steps:
        k, v = rand(g, 4, heads, T, d, dtype=dtype) * amp, rand(g, 4, heads, T, d, dtype=dtype)
        if T > 1:
            grow = [min(4 * page, int(n) + min(x, T)) for n, x in zip(m.lens, counts)]
            bsa.cache_resize(c, i32(*grow))
            assert m.resize(grow) == 0
            counts = [min(x, T, int(n)) for x, n in zip(counts, m.lens)]
        bsa.cache_append(c, k.cuda(), v.cuda(), counts=i32(*counts))
        m.append(k.double().numpy(), v.double().numpy(), counts=counts)
        assert_state(c, m, f"T {T}")
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_append_of_special_values_strides_and_positions(bsa, kind):
    g = torch.Generator().manual_seed(5)
    m = OC.CacheModel(12, 2, 32, 64, 4, 3, kind, 16, seed=3)
    m.resize([70, 40, 96, 20])
    c = upload(bsa, m)
    # Fill, then write into the middle (tokens on both sides stay), rows in
    # [batch, token, head, element] order, sequences in another order, a padded row.
    full = torch.zeros(4, 2, 96, 64, dtype=torch.bfloat16)
    full[:] = rand(g, 4, 2, 96, 64)
    bsa.cache_append(c, full.cuda(), full.cuda(), counts=i32(70, 40, 96, 20), start=i32(0, 0, 0, 0))
    m.append(full.double().numpy(), full.double().numpy(), counts=[70, 40, 96, 20], start=[0] * 4)
    assert_state(c, m)
    x = rand(g, 3, 21, 5, 64)
    x[0, 3, 0, 5], x[0, 4, 1, 6], x[0, 4, 1, 7] = float("nan"), float("inf"), float("-inf")
    x[2, :, :2] = 0.0
    x[2, 0, 0, 0] = 2.0 ** -130
    kk, vv = x[:, :, :2].transpose(1, 2), x[:, :, 2:4].transpose(1, 2)
    xd = x.cuda()
    bsa.cache_append(c, xd[:, :, :2].transpose(1, 2), xd[:, :, 2:4].transpose(1, 2), seqs=i32(2, -1, 0),
                     counts=i32(21, 9, 17), start=i32(11, 4, 33))
    m.append(kk.double().numpy(), vv.double().numpy(), seqs=[2, -1, 0], counts=[21, 9, 17], start=[11, 4, 33])
    assert_state(c, m)
    assert bsa.cache_status(c) == (0, 0)
    # Not stored and reported: past the length, before the start, a bad sequence, a page that is none.
    one = rand(g, 1, 2, 1, 64).cuda()
    for kw, st in ((dict(start=i32(70)), -1), (dict(start=i32(-1)), -1), (dict(seqs=i32(4)), -1),
                   (dict(counts=i32(2)), -1)):
        bsa.cache_append(c, one, one, **kw)
        assert bsa.cache_status(c) == (st, 0), kw
        assert_state(c, m)
    # A sequence named twice: the first row counts.
    two = rand(g, 3, 2, 1, 64)
    bsa.cache_append(c, two.cuda(), two.cuda(), seqs=i32(3, 1, 3))
    m.append(two[:2].double().numpy(), two[:2].double().numpy(), seqs=[3, 1])
    assert bsa.cache_status(c) == (-1, 2)
    assert_state(c, m)
    c.block_table[0, 2] = 12
    bsa.cache_append(c, one, one)
    assert bsa.cache_status(c) == (-7, 0)
    c.block_table[0, 2] = int(m.table[0, 2])
    assert_state(c, m)


# -------------------------------------------------------------- attention

def filled(bsa, lens, heads, page, sb, d, kind, max_pages, seed=0, extra=2):
    """Model and cache with N(0, 1) tokens in sequences of these lengths."""
    g = torch.Generator().manual_seed(seed)
    need = sum(-(-n // page) for n in lens)
    m = OC.CacheModel(need + extra, heads, page, d, len(lens), max_pages, kind, sb, seed=seed)
    rng = np.random.default_rng(seed)
    order = rng.permutation(need + extra)
    at = 0
    for s, n in enumerate(lens):
        h = -(-n // page)
        m.table[s, :h] = order[at:at + h]
        m.refs[order[at:at + h]] = 1
        at += h
        m.lens[s] = n
    T = max(max(lens), 1)
    k = torch.randn(len(lens), heads, T, d, generator=g) * 2.0 ** (torch.rand(len(lens), heads, 1, 1, generator=g) * 4 - 2)
    v = torch.randn(len(lens), heads, T, d, generator=g) * 2.0 ** (torch.rand(len(lens), 1, T, 1, generator=g) * 4 - 2)
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c = upload(bsa, m)
    bsa.cache_append(c, k.cuda(), v.cuda(), counts=i32(*lens), start=i32(*([0] * len(lens))))
    for i in range(2):  # the model takes the GPU's codes (appending has its own tests)
        m.codes[i] = (c.k, c.v)[i].view(torch.uint8).cpu().numpy()
        m.scales[i] = (c.k_scale, c.v_scale)[i].cpu().numpy()
    return m, c


def assert_close(o, lse, ref, q, n_keys, what=""):
    """o, lse of one batch row against the oracle's (O, LSE, A, mag).

    Scores: products of fp16 codes and fp16-exact q in fp32, d + 2 roundings of
    at most 2^-23 (the tensor cores may truncate) of sum |q k|; q below 2^-14
    of its row's largest is off by 2^-25 of that (another 2^-24 of the sum's
    scale); exp2 and its argument 2^-22.  Weights: half an fp16 step, 2^-11, or
    2^-25 of the largest weight where below fp16's normal range; twice the
    scores' error through weight and normalisation.  Output: half a step of its
    type."""
    O, L, A, mag = ref
    d = q.shape[-1]
    ds = mag * (d + 4) * 2.0 ** -23 + 2.0 ** -21
    o64, l64 = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l64), np.isneginf(L)), what
    fin = np.isfinite(L)
    assert not o64[~fin].any(), what
    ulp = torch.finfo(o.dtype).eps / 2
    vmax = np.abs(A).max() + 8 * np.abs(A).max()  # no value is above what 8 of the largest mean holds
    bound = ulp * np.abs(O) + (2.0 ** -11 + 2 * ds[..., None]) * 2 * A + n_keys * 2.0 ** -24 * vmax + 2.0 ** -25
    err = np.abs(o64 - O)
    assert (err <= bound)[fin].all(), (what, float((err / bound)[fin].max()))
    lb = ds + n_keys * 2.0 ** -24 + 2.0 ** -20 + np.abs(np.where(fin, L, 0)) * 2.0 ** -23
    lerr, lb = np.abs(l64[fin] - L[fin]), lb[fin]
    assert (lerr <= lb).all(), (what, float((lerr / lb).max()))


def keep_of(n, nq, Hq, causal=False, mask=None, bk=0):
    j, i = np.arange(n), np.arange(nq)[:, None]
    keep = (j <= n - nq + i) if causal else np.ones((nq, n), bool)
    keep = np.broadcast_to(keep, (Hq, nq, n)).copy()
    if mask is not None:
        sel = np.zeros((Hq, n), bool)
        for h in range(Hq):
            for t in range(n):
                sel[h, t] = t // bk < mask.shape[1] and mask[h, t // bk] != 0
        keep &= sel[:, None]
    return keep


def check_attention(bsa, m, c, q, causal=False, mask=None, bk=0, seqs=None, scale=None, what="", **kw):
    o, lse = bsa.cache_attention(c, q.cuda(), seqs=None if seqs is None else i32(*seqs),
                                 mask=None if mask is None else mask.cuda(), bk=bk, causal=causal, scale=scale, **kw)
    assert bsa.cache_status(c) == (0, 0), what
    for b in range(q.shape[0]):
        s = b if seqs is None else seqs[b]
        if s < 0:
            assert not o[b].any() and torch.isneginf(lse[b]).all(), what
            continue
        k, v = m.values(s)
        keep = keep_of(k.shape[1], q.shape[2], q.shape[1], causal, None if mask is None else mask[b].numpy(), bk)
        ref = OC.attention(q[b].double().numpy(), k, v, keep, scale)
        assert_close(o[b], lse[b], ref, q, k.shape[1], f"{what} row {b}")
    return o, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page,sb,d,g", [(64, 64, 128, 4), (16, 16, 128, 8), (32, 16, 64, 1), (128, 32, 64, 3),
                                         (256, 256, 128, 2)])
def test_single_tokens(bsa, kind, page, sb, d, g):
    lens = [1, 0, 63, 64, 65, 300, 777, 15]
    m, c = filled(bsa, lens, 2, page, sb, d, kind, -(-777 // page), seed=d + page)
    q = rand(torch.Generator().manual_seed(1), len(lens), 2 * g, 1, d)
    check_attention(bsa, m, c, q, what=f"{kind} {page} {sb} {d} {g}")


@pytest.mark.parametrize("nq,g,causal", [(3, 1, True), (2, 8, True), (5, 4, True), (4, 4, False), (17, 3, True),
                                         (33, 4, True), (70, 1, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_several_queries(bsa, nq, g, causal, d):
    # 3 to 132 query rows per K/V head: one or two column tiles, one to four
    # row tiles, several groups; lengths below nq leave rows empty.
    lens = [200, nq, max(1, nq - 2), 500, 0]
    m, c = filled(bsa, lens, 2, 32, 32, d, "e4m3", 16, seed=nq)
    q = rand(torch.Generator().manual_seed(2), len(lens), 2 * g, nq, d)
    check_attention(bsa, m, c, q, causal=causal, what=f"nq {nq} g {g} d {d}")


@pytest.mark.parametrize("bk", [32, 64, 128, 256])
@pytest.mark.parametrize("nq", [1, 4])
def test_block_masks(bsa, bk, nq):
    # Heads of a group select differently, a head selects nothing, a whole group
    # selects nothing, the mask ends before the longest sequence.
    lens = [1000, 130, 640, 1, 0]
    m, c = filled(bsa, lens, 2, 64, 32, 128, "e4m3", 16, seed=bk)
    gen = torch.Generator().manual_seed(bk)
    mask = (torch.rand(5, 8, 900 // bk, generator=gen) < 0.4).to(torch.uint8) * 7
    mask[0, 1], mask[2, 4:] = 0, 0
    q = rand(gen, 5, 8, nq, 128)
    check_attention(bsa, m, c, q, causal=nq > 1, mask=mask, bk=bk, what=f"bk {bk}")


@pytest.mark.parametrize("B,length,heads,g,nq,d,kind", [
    (1, 20000, 1, 2, 1, 64, "int8"), (2, 9000, 4, 2, 1, 64, "int8"), (300, 70, 2, 2, 1, 64, "int8"),
    # tens of tiles per CTA, so that every stage of the ring is used many times
    (6, 24000, 4, 4, 1, 128, "e4m3"), (3, 30000, 4, 12, 1, 128, "int8"), (4, 26000, 4, 4, 6, 64, "e4m3"),
    (2, 24000, 4, 4, 13, 128, "e4m3")])
def test_rows_cut_over_many_ctas(bsa, B, length, heads, g, nq, d, kind):
    lens = [length - (i * 13) % min(length, 61) for i in range(B)]
    m, c = filled(bsa, lens, heads, 64, 64, d, kind, -(-length // 64), seed=B)
    q = rand(torch.Generator().manual_seed(3), B, heads * g, nq, d)
    o, lse = check_attention(bsa, m, c, q, causal=nq > 1, what=f"B {B} length {length}")
    for _ in range(10):  # nothing depends on which CTA is first
        o2, lse2 = bsa.cache_attention(c, q.cuda(), causal=nq > 1)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_masks_of_many_rows(bsa):
    # More (row, head) lists than threads that add them up; empty rows among them.
    B = 210
    lens = [(i * 37) % 91 for i in range(B)]
    m, c = filled(bsa, lens, 2, 32, 32, 128, "e4m3", 3, seed=21)
    gen = torch.Generator().manual_seed(21)
    mask = (torch.rand(B, 4, 3, generator=gen) < 0.5).to(torch.uint8)
    check_attention(bsa, m, c, rand(gen, B, 4, 1, 128), mask=mask, bk=32, what="many rows")


def test_pools_past_32_bit_offsets(bsa):
    """Pages that lie beyond 4 GB in the pools hold and give what the same pages
    of a small cache do."""
    heads, page, d, far = 8, 64, 128, 69000       # 64 KB a page: byte offsets past 2^32
    lens = [700, 130, 64]
    m, c = filled(bsa, lens, heads, page, 32, d, "e4m3", 12, seed=31)
    pages = m.refs.shape[0]
    n = far + pages + 40
    e = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")
    big = bsa.Cache(*(e(n, heads, page, d, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)),
                    *(e(n, heads, page // 32, dtype=torch.float32) for _ in range(2)),
                    torch.where(c.block_table >= 0, c.block_table + far, c.block_table), c.lens.clone(),
                    torch.zeros(n, dtype=torch.int32, device="cuda"))
    big.refs[far:far + pages] = c.refs
    src = torch.arange(pages, dtype=torch.int32, device="cuda")
    bsa.cache_copy_pages(big, c, src + far, src)
    gen = torch.Generator().manual_seed(31)
    new = rand(gen, 3, heads, 1, d).cuda() * 40      # scales grow: old codes are read and rewritten
    q = rand(gen, 3, 2 * heads, 1, d).cuda()
    for x in (c, big):
        bsa.cache_append(x, new, new)
    same = lambda a, b: torch.equal(a[far:far + pages].contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert same(big.k, c.k) and same(big.v, c.v) and same(big.k_scale, c.k_scale) and same(big.v_scale, c.v_scale)
    a, b = bsa.cache_attention(c, q), bsa.cache_attention(big, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    p = bsa.plan(torch.ones(3, 2 * heads, 1, 6, dtype=torch.uint8, device="cuda"), 128, 128, 2)
    q2 = rand(gen, 3, 2 * heads, 128, d).cuda()
    a, b = bsa.cache_forward(p, c, q2, causal=True), bsa.cache_forward(p, big, q2, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bsa.cache_compact(big)                            # back to the front
    assert int((big.refs[:int((c.refs > 0).sum())] > 0).all())
    b = bsa.cache_attention(big, q)
    a = bsa.cache_attention(c, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bsa.cache_status(big) == (0, 0) and bsa.cache_status(c) == (0, 0)


def test_large_and_uneven_scores(bsa):
    # The largest score comes late, scores spread over thousands, scales differ
    # by 2^40 between blocks, q far from 1.
    lens = [700, 700]
    m, c = filled(bsa, lens, 1, 16, 16, 64, "e4m3", 44, seed=9)
    f = torch.exp2(torch.randint(-20, 21, c.v_scale.shape, generator=torch.Generator().manual_seed(1)).float())
    c.v_scale.mul_(f.cuda())
    m.scales[1] = c.v_scale.cpu().numpy()
    last = int(m.table[0, 43])
    c.k_scale[last] *= 512
    m.scales[0] = c.k_scale.cpu().numpy()
    gen = torch.Generator().manual_seed(4)
    for amp, scale in ((1.0, None), (1e4, 1e-4), (2.0 ** -100, 2.0 ** 97)):
        q = (torch.randn(2, 4, 1, 64, generator=gen) * amp).to(torch.bfloat16)
        o, lse = bsa.cache_attention(c, q.cuda(), scale=scale)
        for b in range(2):
            k, v = m.values(b)
            ref = OC.attention(q[b].double().numpy(), k, v, keep_of(700, 1, 4), scale)
            O, L, A, mag = ref
            o64 = o[b].double().cpu().numpy()
            ds = mag * 68 * 2.0 ** -23 + 2.0 ** -21
            # weights under 2^-14 of the largest lose 2^-24 of it, times that key's value
            small = 2.0 ** -24 * np.abs(v).sum(1).max(0)
            bound = 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2 * ds[..., None]) * 2 * A + small
            assert (np.abs(o64 - O) <= bound).all(), (amp, b)
            assert (np.abs(lse[b].double().cpu().numpy() - L) <= ds + 1e-5 + np.abs(L) * 2.0 ** -22).all()


def test_nan_beyond_the_length_and_in_masked_blocks(bsa):
    # What lies in a page past the sequence, and in blocks no head selects, is
    # not attended whatever it holds.
    lens = [100, 70]
    m, c = filled(bsa, lens, 1, 64, 64, 128, "e4m3", 4, seed=6)
    c.k.view(torch.uint8)[int(m.table[0, 1]), :, 36:] = 0x7F
    c.v.view(torch.uint8)[int(m.table[0, 1]), :, 36:] = 0xFF
    gen = torch.Generator().manual_seed(5)
    q = rand(gen, 2, 4, 1, 128)
    check_attention(bsa, m, c, q, what="past the length")
    c.v.view(torch.uint8)[int(m.table[1, 0])] = 0x7F
    mask = torch.ones(2, 4, 2, dtype=torch.uint8)
    mask[1, :, 0] = 0
    m.codes[1][int(m.table[1, 0])] = 0
    check_attention(bsa, m, c, q, mask=mask, bk=64, what="masked block")
    # A NaN that is attended shows in its row.
    o, lse = bsa.cache_attention(c, q.cuda())
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all()


def test_nan_value_masked_for_some_rows_only(bsa):
    # One tile, rows that see different keys: a NaN value reaches only the rows
    # that attend it (the last draft token's value; a block one head selects).
    m, c = filled(bsa, [40], 1, 64, 64, 64, "e4m3", 1, seed=8)
    c.v.view(torch.uint8)[int(m.table[0, 0]), :, 39] = 0x7F
    gen = torch.Generator().manual_seed(7)
    q = rand(gen, 1, 2, 3, 64)
    o, lse = bsa.cache_attention(c, q.cuda(), causal=True)
    assert torch.isnan(o[0, :, 2]).all() and torch.isfinite(lse).all()
    k, v = m.values(0)
    v[:, 39] = 0.0
    ref = OC.attention(q[0].double().numpy(), k, v, keep_of(40, 3, 2, True))
    assert_close(o[0, :, :2], lse[0, :, :2], [x[:, :2] for x in ref], q, 40, "causal NaN")
    mask = torch.ones(1, 2, 2, dtype=torch.uint8)
    mask[0, 0, 1] = 0
    o, lse = bsa.cache_attention(c, q[:, :, :1].cuda(), mask=mask.cuda(), bk=32)
    assert torch.isfinite(o[0, 0]).all() and torch.isnan(o[0, 1]).all()


def test_sequences_padded_rows_strides_types_and_outputs(bsa):
    lens = [150, 20, 333]
    m, c = filled(bsa, lens, 2, 32, 32, 64, "int8", 11, seed=12)
    gen = torch.Generator().manual_seed(6)
    seqs = [2, -1, 0, 2, 1]
    q = torch.randn(5, 3, 6, 64, generator=gen).to(torch.float16).transpose(1, 2)   # [B, Hq = 6, nq = 3, d]
    out = torch.full((5, 3, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.empty(5, 6, 3, device="cuda")
    o, l = bsa.cache_attention(c, q.cuda(), seqs=i32(*seqs), causal=True, out=out[:, :, 1:7].transpose(1, 2), lse=lse)
    assert l.data_ptr() == lse.data_ptr()
    assert (out[:, :, 0] == 7).all() and (out[:, :, 7] == 7).all()
    for b, s in enumerate(seqs):
        if s < 0:
            assert not o[b].any() and torch.isneginf(l[b]).all()
            continue
        k, v = m.values(s)
        ref = OC.attention(q[b].double().numpy(), k, v, keep_of(k.shape[1], 3, 6, True))
        assert_close(o[b], l[b], ref, q, k.shape[1], f"row {b}")


def test_attention_reports_bad_tables_and_sequences(bsa):
    m, c = filled(bsa, [100, 60], 1, 32, 32, 64, "e4m3", 4, seed=1)
    q = rand(torch.Generator().manual_seed(1), 2, 1, 1, 64).cuda()
    good = bsa.cache_attention(c, q)
    c.block_table[1, 1] = 99
    o, lse = bsa.cache_attention(c, q)
    assert bsa.cache_status(c) == (-7, 1)
    assert torch.equal(o[0], good[0][0]) and torch.equal(lse[0], good[1][0])
    o, lse = bsa.cache_attention(c, q, seqs=i32(0, 5))
    assert bsa.cache_status(c) == (-1, 1)
    assert not o[1].any() and torch.isneginf(lse[1]).all() and torch.equal(o[0], good[0][0])


# ---------------------------------------------------------- chunked prefill

@pytest.mark.parametrize("kind,bq,bk,d,page,causal", [("e4m3", 128, 128, 128, 64, True), ("int8", 64, 64, 64, 16, True),
                                                      ("e4m3", 32, 32, 64, 32, False)])
def test_forward_over_the_cache(bsa, kind, bq, bk, d, page, causal):
    lens = [900, 512, 300]
    m, c = filled(bsa, lens, 2, page, 16, d, kind, -(-1024 // page), seed=bq)
    gen = torch.Generator().manual_seed(9)
    Nq, Nk, seqs = 256, 1024, [0, 2, 1, -1]
    mask = (torch.rand(4, 4, Nq // bq, Nk // bk, generator=gen) < 0.6).to(torch.uint8)
    mask[0, 0, 0] = 0
    q = rand(gen, 4, 4, Nq, d)
    p = bsa.plan(mask.cuda(), bq, bk, 2)
    o, lse = bsa.cache_forward(p, c, q.cuda(), seqs=i32(*seqs), causal=causal)
    assert bsa.sync_status(p)[0] == 0 and bsa.cache_status(c) == (0, 0)
    from compare import assert_attention_close
    refs = []
    for b, s in enumerate(seqs):
        if s < 0:
            refs.append((np.zeros((4, Nq, d)), np.full((4, Nq), -np.inf)))
            continue
        k, v = m.values(s)
        n = k.shape[1]
        keep = keep_of(n, Nq, 4, causal)
        keep &= mask[b].numpy().astype(bool).repeat(bq, 1).repeat(bk, 2)[:, :, :n]
        refs.append(OC.attention(q[b].double().numpy(), k, v, keep)[:2])
    assert_attention_close(o, lse, np.stack([r[0] for r in refs]), np.stack([r[1] for r in refs]), f"{kind} {bq} {d}")


@pytest.mark.parametrize("causal", [True, False])
def test_forward_over_the_first_tokens(bsa, causal):
    """A plan of fewer keys than the sequences hold: the queries stay the last
    tokens, so causality leaves out none, some or (300 of 512) more keys."""
    m, c = filled(bsa, [900, 600, 300], 2, 64, 32, 64, "e4m3", 16, seed=44)
    Nq, Nk = 128, 512
    gen = torch.Generator().manual_seed(45)
    mask = (torch.rand(3, 2, 2, 8, generator=gen) < 0.7).to(torch.uint8)
    q = rand(gen, 3, 2, Nq, 64)
    p = bsa.plan(mask.cuda(), 64, 64, 1)
    o, lse = bsa.cache_forward(p, c, q.cuda(), causal=causal)
    assert bsa.sync_status(p)[0] == 0 and bsa.cache_status(c) == (0, 0)
    from compare import assert_attention_close
    refs = []
    for b in range(3):
        k, v = m.values(b)
        n = min(k.shape[1], Nk)
        keep = keep_of(k.shape[1], Nq, 2, causal)[:, :, :n]
        keep &= mask[b].numpy().astype(bool).repeat(64, 1).repeat(64, 2)[:, :, :n]
        refs.append(OC.attention(q[b].double().numpy(), k[:, :n], v[:, :n], keep)[:2])
    assert_attention_close(o, lse, np.stack([r[0] for r in refs]), np.stack([r[1] for r in refs]), f"{causal}")


# ------------------------------------------------------- a run of them together

def test_serving_steps_together_and_captured(bsa):
    """Prefill of a prompt, a fork, decoding steps of both sequences, a dropped
    branch and a compaction; the decoding step captured into a graph and
    replayed gives what the eager calls give."""
    heads, d, page = 2, 64, 32
    m = OC.CacheModel(24, heads, page, d, 3, 8, "e4m3", 16, seed=1)
    c, twin = upload(bsa, m), None
    gen = torch.Generator().manual_seed(2)
    x = rand(gen, 1, heads, 75, d)
    bsa.cache_resize(c, i32(75), i32(0))
    m.resize([75], [0])
    bsa.cache_append(c, x.cuda(), x.cuda(), seqs=i32(0))
    m.append(x.double().numpy(), x.double().numpy(), seqs=[0])
    bsa.cache_fork(c, i32(0), i32(2))
    m.fork([0], [2])
    assert_state(c, m)
    seqs = i32(0, 2)
    new = torch.zeros(2, heads, 1, d, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 2 * heads, 1, d, dtype=torch.bfloat16, device="cuda")
    grown = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 2 * heads, 1, device="cuda")

    def step():
        bsa.cache_resize(c, grown, seqs)
        bsa.cache_append(c, new, new, seqs=seqs)
        bsa.cache_attention(c, q, seqs=seqs, out=out, lse=lse)

    graph = torch.cuda.CUDAGraph()
    for i in range(25):
        kv, qq = rand(gen, 2, heads, 1, d), rand(gen, 2, 2 * heads, 1, d)
        new.copy_(kv)
        q.copy_(qq)
        grown.copy_(i32(76 + i, 76 + i))
        if i == 3:
            with torch.cuda.graph(graph):
                step()
        if i < 3:
            step()
        else:
            graph.replay()
        m.resize([76 + i, 76 + i], [0, 2])
        m.append(kv.double().numpy(), kv.double().numpy(), seqs=[0, 2])
        assert_state(c, m, f"step {i}")
        if i % 8 == 0:
            for b, s in enumerate((0, 2)):
                k, v = m.values(s)
                ref = OC.attention(qq[b].double().numpy(), k, v, keep_of(76 + i, 1, 2 * heads))
                assert_close(out[b], lse[b], ref, qq, 76 + i, f"step {i} row {b}")
    bsa.cache_free(c, i32(0))
    m.resize([0], [0])
    bsa.cache_compact(c)
    m.compact()
    assert_state(c, m)
    graph.replay()  # the captured step again: sequence 0 from empty to 100 tokens, 2 unchanged
    torch.cuda.synchronize()
    assert bsa.cache_status(c) == (0, 0)


def test_two_streams_read_one_cache(bsa):
    m, c = filled(bsa, [3000, 2000, 10], 4, 64, 64, 128, "e4m3", 47, seed=3)
    gen = torch.Generator().manual_seed(3)
    q1, q2 = rand(gen, 3, 16, 1, 128).cuda(), rand(gen, 3, 16, 2, 128).cuda()
    a, b = bsa.cache_attention(c, q1), bsa.cache_attention(c, q2, causal=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((bsa.cache_attention(c, q1, stream=s1), bsa.cache_attention(c, q2, causal=True, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], a[0]) and torch.equal(x[1], a[1])
        assert torch.equal(y[0], b[0]) and torch.equal(y[1], b[1])


def test_calls_on_another_stream_use_memory_of_their_own(bsa):
    """Results and scratch of calls on a given stream are that stream's memory:
    work that is still queued on the current stream cannot run into them."""
    m, c = filled(bsa, [2500, 700], 2, 64, 64, 64, "int8", 40, seed=4)
    gen = torch.Generator().manual_seed(4)
    q = rand(gen, 2, 8, 1, 64).cuda()
    want = bsa.cache_attention(c, q)
    p = bsa.plan(torch.ones(2, 8, 1, 20, dtype=torch.uint8, device="cuda"), 128, 128, 4)
    q2 = rand(gen, 2, 8, 128, 64).cuda()
    want2 = bsa.cache_forward(p, c, q2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        busy = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        for _ in range(20):
            busy.fill_(255)          # queued on the current stream ...
        del busy                     # ... whose memory is free to be handed out there
        got, got2 = bsa.cache_attention(c, q, stream=side), bsa.cache_forward(p, c, q2, stream=side)
        torch.cuda.synchronize()
        for x, y in zip(got + got2, want + want2):
            assert torch.equal(x, y)


def test_scratch_of_the_default_stream_is_its_own(bsa):
    """A first call on the (given) default stream, from another current stream
    with work under way on memory that it has given back: the scratch that
    default-stream calls share must not be that memory."""
    m, c = filled(bsa, [700, 30], 2, 64, 64, 128, "e4m3", 12, seed=31)
    q = rand(torch.Generator().manual_seed(32), 2, 8, 1, 128).cuda()
    want = bsa.cache_attention(c, q)
    torch.cuda.synchronize()
    from block_sparse_attention_plan_gb300 import _cache
    was, _cache._kept = _cache._kept, {}
    try:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            back = torch.empty(_cache._KEPT_BYTES, dtype=torch.uint8, device="cuda")
            at = back.data_ptr()
            del back
            bsa.cache_attention(c, q, stream=torch.cuda.default_stream())
        torch.cuda.synchronize()
        assert _cache._kept[c.device.index].data_ptr() != at
    finally:
        _cache._kept = was
    got = bsa.cache_attention(c, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_threads_on_the_default_stream(bsa):
    """Calls of two host threads on one stream share their scratch in turn."""
    import threading
    m, c = filled(bsa, [3000, 1500, 40], 2, 64, 64, 64, "e4m3", 47, seed=14)
    gen = torch.Generator().manual_seed(14)
    qs = [rand(gen, 3, 8, n, 64).cuda() for n in (1, 3)]
    want = [bsa.cache_attention(c, q) for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            for _ in range(200):
                got = bsa.cache_attention(c, qs[i])
                if not (torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])):
                    bad.append(i)
        except Exception as e:  # (a thread's own does not fail the test)
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]


def test_growth_past_32_bits_of_pages_is_refused(bsa):
    # 64 sequences of 2^26 pages each: 2^32 in all, for a pool of 8.
    c = bsa.cache_create(8, 1, 16, 64, 64, 1 << 26)
    bsa.cache_resize(c, i32(40), i32(5))
    bsa.cache_resize(c, torch.full((64,), 1 << 30, dtype=torch.int32, device="cuda"))
    assert bsa.cache_status(c) == (-5, (1 << 31) - 1 - 5)
    assert c.lens.tolist() == [0] * 5 + [40] + [0] * 58 and c.refs.tolist() == [1] * 3 + [0] * 5
    assert c.block_table[5, :4].tolist() == [0, 1, 2, -1] and int(c.block_table[6].max()) == -1


@pytest.mark.parametrize("kind", KINDS)
def test_append_rounds_once_at_scales_of_others(bsa, kind):
    """Scales that are no powers of two, where fp32 would round code * was /
    scale, or x / scale, to a tie that the exact value is not."""
    ratio = {}  # odd codes c, ratios r in [1/2, 1): c r is not, but rounds to, k + 1/2
    for c in range(5, 127, 2):
        for k in range(c // 2, c):
            r = np.float32((k + 0.5) / c)
            if 0.5 <= r < 1 and float(r) * c != k + 0.5 and np.float32(r * np.float32(c)) == k + 0.5:
                ratio[float(r)] = c
    ratios = np.array(sorted(ratio), np.float32)[:128]
    assert len(ratios) == 128
    m = OC.CacheModel(128, 1, 16, 128, 128, 1, kind, seed=3)
    assert m.resize([16] * 128) == 0
    vals = np.arange(1, 128) if kind == "int8" else np.arange(1, 0x7f)
    for w in range(2):  # every code, either sign, at a scale that grows to 1
        m.codes[w][..., :len(vals)] = vals.astype(np.uint8)
        m.codes[w][:, :, 8:, :len(vals)] = (-vals).astype(np.int8).view(np.uint8) if kind == "int8" else vals + 0x80
        m.scales[w][m.table[:, 0], 0, 0] = ratios
    c = upload(bsa, m)
    x = torch.full((128, 1, 1, 128), 1.0 * OC.TOP[kind]).to(torch.bfloat16)
    m.append(x.double().numpy(), x.double().numpy(), range(128), None, [5] * 128)
    bsa.cache_append(c, x.cuda(), x.cuda(), start=i32(*[5] * 128))
    assert (m.scales[0][m.table[:, 0]] == 1).all()
    assert_state(c, m)
    # x / scale, the scale kept: every bf16 number from 2^-3 to 2^5 on each scale in [1/2, 1).
    m.scales[0][m.table[:, 0], 0, 0] = m.scales[1][m.table[:, 0], 0, 0] = ratios
    c = upload(bsa, m)
    x = (torch.arange(1024, dtype=torch.int16) + 0x3e00).view(torch.bfloat16).reshape(1, 1, 8, 128).repeat(128, 1, 1, 1)
    m.append(x.double().numpy(), -x.double().numpy(), range(128), None, [0] * 128)
    bsa.cache_append(c, x.cuda(), -x.cuda(), start=i32(*[0] * 128))
    assert_state(c, m)
    assert bsa.cache_status(c) == (0, 0)


def test_append_leaves_shared_pages_alone(bsa):
    gen = torch.Generator().manual_seed(71)
    m = OC.CacheModel(12, 2, 16, 64, 4, 4, seed=7)
    assert m.resize([20], [0]) == 0
    c = upload(bsa, m)

    def append(T, seqs, start=None):
        k, v = (rand(gen, len(seqs), 2, T, 64) for _ in range(2))
        m.append(k.double().numpy(), v.double().numpy(), seqs, None, start)
        bsa.cache_append(c, k.cuda(), v.cuda(), seqs=i32(*seqs), start=None if start is None else i32(*start))
        assert_state(c, m)

    append(20, [0])
    assert bsa.cache_status(c) == (0, 0)
    bsa.cache_fork(c, i32(0), i32(2))
    m.fork([0], [2])
    # Both hold pages of tokens 0 .. 19: nothing of either row is stored.
    append(3, [0, 2])
    assert bsa.cache_status(c)[0] == -1
    # Grown by 14, sequence 2 has tokens 16 .. 33 to itself, and 0 (alone with
    # its last page again) 16 .. 19; tokens 0 .. 15 stay as they are.
    bsa.cache_resize(c, i32(34), i32(2))
    assert m.resize([34], [2]) == 0
    append(14, [2])
    append(4, [0])
    assert bsa.cache_status(c) == (0, 0)
    append(20, [2], [8])  # 8 .. 15 lie in the shared page, 16 .. 27 do not
    assert bsa.cache_status(c) == (-1, 0)


def test_free_of_every_sequence(bsa):
    c = bsa.cache_create(64, 1, 16, 64, 5000, 2)
    bsa.cache_resize(c, torch.full((60,), 16, dtype=torch.int32, device="cuda"))
    assert int((c.refs > 0).sum()) == 60
    bsa.cache_free(c)
    assert bsa.cache_status(c) == (0, 0)
    assert not c.refs.any() and not c.lens.any() and (c.block_table == -1).all()


def test_argument_errors(bsa):
    m, c = filled(bsa, [10], 2, 32, 32, 64, "e4m3", 1, seed=3)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (q[..., :32], q.float(), q.cpu(), q[0]):
        with pytest.raises((ValueError, bsa.BsaError)):
            bsa.cache_attention(c, bad)
    with pytest.raises(bsa.BsaError) as e:
        bsa.cache_attention(c, q[:, :3])                       # 3 query heads over 2
    assert e.value.status == -1
    with pytest.raises(bsa.BsaError) as e:
        bsa.cache_attention(c, q, mask=torch.ones(1, 4, 1, dtype=torch.uint8, device="cuda"), bk=48)
    assert e.value.status == -2
    with pytest.raises(bsa.BsaError):
        bsa.cache_attention(c, torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda"))  # 2 rows, 1 sequence
    with pytest.raises(bsa.BsaError):
        bsa.cache_attention(c, q, scale=float("nan"))
    with pytest.raises(ValueError):
        bsa.cache_attention(c, q, seqs=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        bsa.cache_append(c, q, q)                              # 4 heads
    with pytest.raises(bsa.BsaError):
        bsa.cache_append(c, *(torch.zeros(1, 2, 33, 64, dtype=torch.bfloat16, device="cuda"),) * 2)  # over a sequence
    with pytest.raises(bsa.BsaError):                          # rows that start off a 16-byte boundary
        x = torch.zeros(1, 2, 1, 72, dtype=torch.bfloat16, device="cuda")[..., 4:68]
        bsa.cache_append(c, x, x)
    with pytest.raises(ValueError):
        bsa.cache_attention(c, q, mask=torch.ones(1, 4, 0, dtype=torch.uint8, device="cuda"), bk=64)
    for bad in (dict(page_size=24), dict(page_size=8), dict(page_size=512), dict(d=96), dict(scale_block=8)):
        with pytest.raises((bsa.BsaError, ValueError)):
            bsa.cache_create(**{**dict(num_pages=4, heads=1, page_size=32, d=64, max_seqs=1, max_pages=1), **bad})
    with pytest.raises(bsa.BsaError):
        bsa.cache_free(c, torch.full((5000,), -1, dtype=torch.int32, device="cuda"))
    w = torch.ones(1, 4, 2, 4, dtype=torch.uint8, device="cuda")
    with pytest.raises(bsa.BsaError) as e:
        p = bsa.plan(w, 64, 64, 2, flags=bsa.PLAN_Q64)
        bsa.cache_forward(p, c, torch.zeros(1, 4, 128, 64, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(bsa.BsaError) as e:
        p = bsa.plan(w, 64, 64, 1)
        bsa.cache_forward(p, c, torch.zeros(1, 4, 128, 64, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == -7                                # 4 K/V heads against 2
    assert bsa.cache_status(c) == (0, 0)
