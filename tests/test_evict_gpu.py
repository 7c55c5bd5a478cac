"""GPU tests of the cache's gathered weights (bsa_cache_weigh, against fp64 with
bounds from the arithmetic) and of eviction by them (bsa_cache_evict, bit for bit
against the oracle's model)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as OC

pytestmark = pytest.mark.gpu

KINDS = ["e4m3", "int8"]


def upload(bsa, m, device="cuda"):
    dt = torch.float8_e4m3fn if m.kind == "e4m3" else torch.int8
    t = lambda a: torch.from_numpy(a.copy()).to(device)
    return bsa.Cache(*(t(x).view(dt) for x in m.codes), *(t(x) for x in m.scales), t(m.table), t(m.lens), t(m.refs))


def assert_state(c, m, what=""):
    for name, got, want in (("table", c.block_table, m.table), ("lens", c.lens, m.lens), ("refs", c.refs, m.refs),
                            ("k", c.k.view(torch.uint8), m.codes[0]), ("v", c.v.view(torch.uint8), m.codes[1]),
                            ("k_scale", c.k_scale, m.scales[0]), ("v_scale", c.v_scale, m.scales[1])):
        same = np.array_equal(got.cpu().numpy(), want, equal_nan=want.dtype.kind == "f")
        assert same, (what, name)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(kind, lens, H, page, sb, d, seed=0, spare=3, width=None):
    """A model whose sequences hold tokens of blocks of several magnitudes, in shuffled pages."""
    rng = np.random.default_rng(seed)
    held = [-(-n // page) for n in lens]
    m = OC.CacheModel(sum(held) + spare, H, page, d, len(lens), width or max(max(held), 1), kind, sb, seed=seed)
    perm = rng.permutation(sum(held) + spare)
    at = 0
    for s, n in enumerate(held):
        m.table[s, :n] = perm[at:at + n]
        m.refs[perm[at:at + n]] = 1
        at += n
    m.lens[:] = lens
    for w in range(2):
        top = 0x7E if kind == "e4m3" else 0x7F
        code = rng.integers(0, top, m.codes[w].shape).astype(np.uint8)
        m.codes[w] = code | (rng.integers(0, 2, code.shape).astype(np.uint8) << 7) if kind == "e4m3" else np.where(
            rng.random(code.shape) < 0.5, code, (-code.astype(np.int8)).view(np.uint8))
        m.scales[w] = (2.0 ** rng.integers(-9, -6, m.scales[w].shape)).astype(np.float32)
    return m


# ------------------------------------------------------------------ weights

def weigh_both(bsa, m, c, q, lse, w0, seqs=None, mask=None, bk=0, causal=False, fresh=0):
    """The kernel's weights against the oracle's: each exponential's argument is off by the score's error (the row
    rounded to fp16: 2^-25 of its largest element times sum |k|; fp32 sums of exact products: under 2^-16 sum |q k|,
    128 terms of 2^-23) and by 2^-22 of its terms; ex2 by 2^-22; sums of the rows by 2^-23 each."""
    B, Hq, nq, d = q.shape
    g = Hq // w0.shape[1]
    n = max(int(x) for x in m.lens)
    lens = [int(m.lens[b if seqs is None else seqs[b]]) if seqs is None or seqs[b] >= 0 else 0 for b in range(B)]

    def keep(b, h, i, j):
        if causal and j > lens[b] - nq + i:
            return False
        return mask is None or (j // bk < mask.shape[2] and mask[b, h, j // bk] != 0)

    qd, ld = q.double().numpy(), lse.double().numpy()
    want = w0.double().numpy().copy()
    m.weigh(want, qd, ld, seqs=seqs, keep=keep if causal or mask is not None else None, fresh=fresh)
    w = w0.cuda()
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), w, seqs=None if seqs is None else i32(*seqs),
                    mask=None if mask is None else torch.from_numpy(mask).cuda(), bk=bk, causal=causal, fresh=fresh)
    got = w.double().cpu().numpy()
    tol = np.zeros_like(want)
    for b in range(B):
        s = b if seqs is None else seqs[b]
        if s < 0:
            continue
        k = m.values(s)[0]
        for h in range(Hq):
            kk = k[h // g]
            for i in range(nq):
                z = ld[b, h, i]
                if z == -math.inf:
                    continue
                x = qd[b, h, i]
                sc = kk @ x / math.sqrt(d)
                err = (2.0 ** -16 * (np.abs(kk) @ np.abs(x)) + 2.0 ** -24 * np.abs(x).max() * np.abs(kk).sum(1)) / math.sqrt(d) \
                    + 2.0 ** -22 * (np.abs(sc) + abs(z) + 1)
                tol[s, h // g, :lens[b]] += np.exp(sc - z) * np.expm1(err)
    tol += 2.0 ** -23 * (g * nq + 2) * np.abs(want) + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    for s in range(want.shape[0]):  # rows of no call, and weights behind the last token, are left as they were
        if s not in (range(B) if seqs is None else seqs):
            assert np.array_equal(got[s], w0[s].double().numpy())
    assert not bad.any(), (np.abs(got - want)[bad].max(), np.argwhere(bad)[:4])
    return w


@pytest.mark.parametrize("kind,page,sb,d,lens,Hkv,g,nq,causal,bk,fresh", [
    ("e4m3", 64, 64, 128, [1, 0, 37, 300], 2, 4, 1, False, 0, 1),
    ("int8", 16, 16, 64, [65, 130, 7], 2, 1, 1, False, 0, 0),
    ("e4m3", 128, 16, 64, [200, 64], 1, 7, 3, True, 0, 3),
    ("int8", 32, 32, 128, [100, 2, 33], 1, 8, 5, True, 0, 1 << 30),   # fewer tokens than queries
    ("e4m3", 16, 16, 128, [90, 33], 1, 4, 40, True, 0, 1 << 30),      # 160 rows: two passes
    ("e4m3", 64, 32, 64, [500, 131], 2, 3, 1, False, 32, 1),          # two blocks in a tile
    ("int8", 64, 64, 128, [500, 131], 2, 3, 2, True, 64, 500),        # fresh tokens in blocks of no head
    ("e4m3", 256, 64, 64, [700], 1, 40, 1, False, 128, 1),            # more heads of a group than lanes
    ("int8", 16, 16, 64, [260], 1, 5, 30, False, 32, 0)])
def test_weights_against_the_oracle(bsa, kind, page, sb, d, lens, Hkv, g, nq, causal, bk, fresh):
    gen = torch.Generator().manual_seed(sum(lens) + d)
    m = filled(kind, lens, Hkv, page, sb, d, seed=5)
    for s in m.scales:  # scores of a few units
        s *= np.float32(0.25)
    c = upload(bsa, m)
    B = len(lens)
    q = (torch.randn(B, Hkv * g, nq, d, generator=gen) * 0.5).to(torch.float16 if page == 32 else torch.bfloat16)
    lse = torch.randn(B, Hkv * g, nq, generator=gen) + 3
    lse[0, -1, 0] = -math.inf
    w0 = torch.rand(B, Hkv, m.table.shape[1] * page, generator=gen)
    mask = None
    if bk:
        mask = (np.random.default_rng(1).random((B, Hkv * g, max(1, max(lens) // bk))) < 0.3).astype(np.uint8) * 5
    weigh_both(bsa, m, c, q, lse, w0, mask=mask, bk=bk, causal=causal, fresh=fresh)
    assert bsa.cache_status(c) == (0, 0)


def test_weights_of_listed_sequences(bsa):
    gen = torch.Generator().manual_seed(9)
    m = filled("e4m3", [70, 0, 130, 64], 2, 32, 32, 64, seed=6)
    c = upload(bsa, m)
    q = (torch.randn(4, 4, 1, 64, generator=gen) * 0.2).to(torch.bfloat16)
    lse = torch.zeros(4, 4, 1)
    w0 = torch.rand(4, 2, 160, generator=gen)
    want = weigh_both(bsa, m, c, q, lse, w0, seqs=[2, -1, 0, 1], fresh=1)
    assert bsa.cache_status(c) == (0, 0)
    # named again: skipped and recorded; out of range: recorded
    w = w0.cuda()
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), w, seqs=i32(2, 2, 0, 2))
    assert bsa.cache_status(c)[0] == -1
    assert torch.equal(w[2], want[2])
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), w, seqs=i32(-1, 4, -1, -1))
    assert bsa.cache_status(c) == (-1, 1)
    # no room for the sequence's weights
    narrow = torch.ones(4, 2, 100, device="cuda")
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), narrow)
    assert bsa.cache_status(c) == (-1, 2) and (narrow[2] == 1).all() and (narrow[0, :, :69] > 1).all()
    # strided queries, and ones that repeat
    t = torch.zeros(4, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    t.copy_(q.transpose(1, 2))
    a, b = w0.cuda(), w0.cuda()
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), a)
    bsa.cache_weigh(c, t.transpose(1, 2), lse.cuda(), b)
    assert torch.equal(a, b)
    bsa.cache_weigh(c, q[:1].cuda().expand(4, 4, 1, 64), lse.cuda(), b)
    assert bsa.cache_status(c) == (0, 0)


def test_weights_of_tokens_in_no_page(bsa):
    m = filled("int8", [100], 1, 16, 16, 128, seed=7)
    m.table[0, 2], m.table[0, 4] = -1, 99
    c = upload(bsa, m)
    w = torch.ones(1, 1, 112, device="cuda")
    bsa.cache_weigh(c, torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 4, 1, device="cuda"), w, fresh=40)
    assert bsa.cache_status(c) == (-7, 0)
    want = np.full(112, 5.0)         # four rows of weight exp(0)
    want[60:100] = 4
    want[32:48], want[64:80] = 1, 0  # as they were; fresh
    want[100:] = 1
    assert np.array_equal(w[0, 0].cpu().numpy(), want)


def test_nan_and_infinities_stay_with_their_tokens(bsa):
    m = filled("e4m3", [50], 1, 64, 16, 128, seed=8)
    m.codes[0][m.table[0, 0], 0, 50:] = 0x7F  # behind the last token
    m.codes[0][m.table[0, 0], 0, 20] = 0x7F
    m.scales[0][m.table[0, 0], 0, 2] = math.inf
    c = upload(bsa, m)
    w = torch.zeros(1, 1, 64, device="cuda")
    q = torch.ones(1, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    bsa.cache_weigh(c, q, torch.full((1, 2, 1), 50.0, device="cuda"), w)
    bad = ~torch.isfinite(w[0, 0].cpu())
    assert bad[20] and not bad[:20].any() and not bad[21:32].any() and not bad[48:].any() and (w[0, 0, 50:] == 0).all()


@pytest.mark.parametrize("g,nq", [(4, 1), (3, 7), (8, 20)])
def test_a_row_without_a_sum_gives_nothing_whatever_it_holds(bsa, g, nq):
    gen = torch.Generator().manual_seed(g)
    m = filled("e4m3", [75, 40], 2, 32, 32, 128, seed=8)
    q = (torch.randn(2, 2 * g, nq, 128, generator=gen) * 0.2).to(torch.bfloat16)
    lse = torch.randn(2, 2 * g, nq, generator=gen) + 3
    lse[0, 1, -1] = lse[1, 0, 0] = lse[1, g, 0] = -math.inf
    w0 = torch.rand(2, 2, 96, generator=gen)
    plain = w0.cuda()
    bsa.cache_weigh(upload(bsa, m), q.cuda(), lse.cuda(), plain, fresh=0)
    q[0, 1, -1] = math.inf
    q[1, 0, 0, 5] = math.nan
    q[1, g, 0, ::2] = -math.inf
    got = w0.cuda()
    bsa.cache_weigh(upload(bsa, m), q.cuda(), lse.cuda(), got, fresh=0)
    assert plain.isfinite().all() and torch.equal(plain, got)


@pytest.mark.parametrize("kind,d", [("e4m3", 128), ("int8", 64)])
def test_weights_of_a_batch_in_one_line(bsa, kind, d):
    """Many pairs cut over all CTAs: uneven lengths, several tiles a warp, against torch in fp64."""
    lens = [(i * 377) % 2900 for i in range(40)]
    m = filled(kind, lens, 3, 32, 16, d, seed=9, width=100)
    for s in m.scales:
        s *= np.float32(0.25)
    c = upload(bsa, m)
    gen = torch.Generator().manual_seed(2)
    q = (torch.randn(40, 6, 1, d, generator=gen) * 0.3).to(torch.bfloat16)
    lse = torch.randn(40, 6, 1, generator=gen) + 5
    w0 = torch.rand(40, 3, 3200, generator=gen)
    weigh_both(bsa, m, c, q, lse, w0, fresh=1)
    a, b = w0.cuda(), w0.cuda()
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), a)
    bsa.cache_weigh(c, q.cuda(), lse.cuda(), b)
    assert torch.equal(a, b)  # the same bits every time


# ------------------------------------------------------------------ eviction

def evict_both(bsa, m, c, w0, keep, seqs=None, sink=0, recent=0, keep_max=None):
    heads = w0.shape[1]
    ref = w0.numpy().copy()
    rows = m.evict(ref, keep, seqs=seqs, sink=sink, recent=recent)
    w = w0.cuda()
    kept = torch.full((len(keep), heads, keep_max or w0.shape[2]), -7, dtype=torch.int32, device="cuda")
    got = bsa.cache_evict(c, w, i32(*keep), seqs=None if seqs is None else i32(*seqs), sink=sink, recent=recent, kept=kept)
    assert got is kept
    assert_state(c, m)
    assert np.array_equal(w.cpu().numpy(), ref, equal_nan=True)
    k = kept.cpu().numpy()
    for i, r in enumerate(rows):
        for h in range(heads):
            want = [] if r is None else r[h][:k.shape[2]]
            assert list(k[i, h, :len(want)]) == want and (k[i, h, len(want):] == -7).all(), (i, h)
    return w


def heavy(gen, *shape):
    w = torch.exp(2 * torch.randn(*shape, generator=gen))
    return torch.where(torch.rand(*shape, generator=gen) < 0.2, 0.0, w)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page,sb,d,lens,keep,sink,recent", [
    (16, 16, 64, [1, 0, 40, 100], [1, 0, 16, 33], 0, 0),
    (64, 16, 128, [130, 64, 65], [64, 63, 0], 4, 10),
    (64, 64, 128, [500, 7, 300], [300, 3, 299], 2, 3),
    (128, 32, 64, [700, 640], [257, 128], 1000, 5),     # more sinks than budget
    (256, 256, 128, [900], [513], 3, 1000),             # more recent ones than budget
    (32, 16, 64, [2100, 3000], [1100, 2999], 16, 64),   # several rounds
    (16, 16, 128, [5000], [4500], 0, 0)])
def test_eviction_against_the_model(bsa, kind, page, sb, d, lens, keep, sink, recent):
    gen = torch.Generator().manual_seed(sum(lens))
    m = filled(kind, lens, 2, page, sb, d, seed=3)
    c = upload(bsa, m)
    w = heavy(gen, len(lens), 2, m.table.shape[1] * page)
    w = evict_both(bsa, m, c, w, keep, sink=sink, recent=recent)
    assert bsa.cache_status(c) == (0, 0)
    # again, to smaller budgets; then nothing more to do
    small = [k // 2 for k in keep]
    w = evict_both(bsa, m, c, w.cpu(), small, sink=1, recent=2)
    evict_both(bsa, m, c, w.cpu(), small)
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("lens,keep,H,page", [
    ([100000], [3001], 2, 256),                     # shares of a cluster's CTAs
    ([400007], [2500], 1, 256),                     # longer than a cluster holds
    ([50001] + [9] * 310, [2000] + [4] * 310, 1, 64)])  # a CTA each, one with more than it holds
def test_long_sequences(bsa, lens, keep, H, page):
    m = filled("int8", lens, H, page, 16, 64, seed=6)
    c = upload(bsa, m)
    w = heavy(torch.Generator().manual_seed(1), len(lens), H, m.table.shape[1] * page)
    w[0, 0, :5000] = 1.0                            # ties over the border of shares
    w[0, 0, 20000:45000] = 1.0
    evict_both(bsa, m, c, w, keep, sink=3, recent=5, keep_max=max(keep))
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_ties_zeros_nan_and_negative_weights(bsa, kind):
    rng = np.random.default_rng(4)
    m = filled(kind, [3000, 3000, 3000, 3000], 1, 64, 16, 64, seed=1)
    c = upload(bsa, m)
    w = np.zeros((4, 1, 3008), np.float32)
    w[1] = rng.choice([0.0, -0.0, 1.0, 2.0, 2.0 + 2.0 ** -22], w[1].shape)
    w[2] = rng.choice([math.nan, -1.0, 0.0, -math.inf, math.inf, 1e-45, 3.0], w[2].shape)
    w[3] = 1.0 + rng.integers(0, 40, w[3].shape) * np.float32(2.0 ** -23)  # the last digit decides
    evict_both(bsa, m, c, torch.from_numpy(w), [1000, 1700, 2500, 800], sink=3, recent=100)
    assert bsa.cache_status(c) == (0, 0)


def test_scales_that_are_none_and_no_powers_of_two(bsa):
    m = filled("e4m3", [256], 2, 64, 16, 128, seed=2)
    rng = np.random.default_rng(0)
    for s in m.scales:
        s[:] = 2.0 ** rng.integers(-9, -6, s.shape)
        s[m.table[0, 0], 0, :] = [0.0, math.nan, math.inf, -1.0]
        s[m.table[0, 1], 1, :2] = 0.0
    c = upload(bsa, m)
    w = heavy(torch.Generator().manual_seed(1), 1, 2, 256)
    evict_both(bsa, m, c, w, [100])
    assert bsa.cache_status(c) == (0, 0)
    # Scales that are no powers of two: the ratio is rounded to fp32, the product once more, to the code
    m = filled("int8", [200], 1, 16, 16, 64, seed=2)
    for s in m.scales:
        s[:] = (rng.random(s.shape) + 0.5).astype(np.float32)
    c = upload(bsa, m)
    before = c.k.float().clone(), c.k_scale.clone(), c.block_table.clone()
    kept = bsa.cache_evict(c, torch.rand(1, 1, 208, device="cuda"), i32(50))[0, 0, :50].long()
    page = lambda j: before[2][0, j // 16].long()
    x = before[0][page(kept), 0, kept % 16] * before[1][page(kept), 0, 0].unsqueeze(1)
    to = torch.arange(50, device="cuda")
    sc = c.k_scale[c.block_table[0, to // 16].long(), 0, 0].unsqueeze(1)
    y = c.k[c.block_table[0, to // 16].long(), 0, to % 16].float() * sc
    assert ((x - y).abs() <= sc * (0.5 + 2.0 ** -15)).all()  # half a step of the code, and the ratio's 127 * 2^-23
    assert torch.equal(sc.view(-1)[:48].view(3, 16)[:, 0], before[1][page(kept), 0, 0][:48].view(3, 16).amax(1))


def test_listed_sequences_and_bad_items(bsa):
    gen = torch.Generator().manual_seed(1)
    lens = [100, 80, 0, 60, 90]
    m = filled("int8", lens, 2, 16, 16, 64, seed=4, spare=10)
    c = upload(bsa, m)
    w = heavy(gen, 5, 2, 112)
    w = evict_both(bsa, m, c, w, [50, 9, 40], seqs=[4, -1, 0], sink=2, recent=5, keep_max=60)
    assert bsa.cache_status(c) == (0, 0)

    def skipped(keep, seqs, status, weights=w, keep_max=60, **kw):
        t = weights.clone()
        kept = torch.full((len(keep), 2, keep_max), -7, dtype=torch.int32, device="cuda")
        bsa.cache_evict(c, t, i32(*keep), seqs=i32(*seqs), kept=kept, **kw)
        assert bsa.cache_status(c) == status
        assert_state(c, m)
        assert torch.equal(t, weights)
        return kept

    skipped([5, -1], [2, 3], (-1, 1))                     # a budget below 0
    skipped([5], [9], (-1, 0))                            # no such sequence
    skipped([10], [3], (-1, 0), keep_max=9)               # no room for the list
    skipped([10], [3], (-1, 0), weights=w[:, :, :50].contiguous())  # nor for the weights
    kept = skipped([200, 70], [3, 1], (-1, 1))            # not cut; cut to more than there is room for
    assert list(kept[0, 0].cpu()) == list(range(60)) and (kept[1] == -7).all()
    # a later row that names a sequence again
    ref = w.cpu().numpy().copy()
    m.evict(ref, [30], seqs=[3])
    t = w.clone()
    bsa.cache_evict(c, t, i32(30, 20), seqs=i32(3, 3))
    assert bsa.cache_status(c) == (-1, 1)
    assert_state(c, m)
    assert np.array_equal(t.cpu().numpy(), ref)
    # a token in no page
    good = m.table[1, 3]
    for bad in (-1, 1000):
        m.table[1, 3] = bad
        c.block_table[1, 3] = bad
        skipped([10], [1], (-7, 1))
    m.table[1, 3] = good
    c.block_table[1, 3] = int(good)


def test_pages_that_other_sequences_hold(bsa):
    m = filled("e4m3", [100, 0], 1, 16, 16, 64, seed=4, spare=10)
    c = upload(bsa, m)
    w = heavy(torch.Generator().manual_seed(5), 2, 1, 112)
    bsa.cache_fork(c, i32(0), i32(1))
    m.fork([0], [1])
    t = w.cuda()
    bsa.cache_evict(c, t, i32(40), seqs=i32(1))
    assert bsa.cache_status(c) == (-1, 0)
    assert_state(c, m)
    # shared pages that are only given back are no hindrance
    for j in range(3):  # the first three become the sequence's own
        m.refs[m.table[0, j]] -= 1
        p = int(np.nonzero(m.refs == 0)[0][0])
        m.refs[p], m.table[1, j] = 1, p
    c.block_table.copy_(torch.from_numpy(m.table))
    c.refs.copy_(torch.from_numpy(m.refs))
    for x in m.codes + m.scales:
        for j in range(3):
            x[m.table[1, j]] = x[m.table[0, j]]
    c = upload(bsa, m)
    evict_both(bsa, m, c, w, [100, 48], recent=4)
    assert bsa.cache_status(c) == (0, 0) and m.refs.max() == 1


@pytest.mark.parametrize("kind", KINDS)
def test_a_pool_past_32_bit_offsets(bsa, kind):
    """Pages, scales and weights whose offsets in bytes (and elements) pass 2^32."""
    page, d, H = 256, 128, 8
    pages = (1 << 32) // (page * d * H) + 40
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    pool = lambda: torch.randint(0, 100, (pages, H, page, d), dtype=torch.uint8, device="cuda").view(dt)
    k, v = pool(), pool()
    scale = torch.full((pages, H, page // 16), 2.0 ** -8, device="cuda")
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    table[1, :4] = torch.tensor([pages - 1, 3, pages - 7, pages - 2])
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[1, :4].long()] = 1
    lens = i32(0, 1000)
    c = bsa.Cache(k, v, scale, scale.clone(), table, lens, refs)
    w = torch.rand(2, H, (1 << 28) + 5, device="cuda")   # the second sequence's begin past 2^31 elements
    q = torch.randn(1, 16, 1, d, device="cuda").to(torch.bfloat16)
    own = k.view(torch.uint8)[table[1, :4].long()].clone()           # [4, H, page, d]
    keys = own.view(dt).float().permute(1, 0, 2, 3).reshape(H, 1024, d)[:, :1000] * 2.0 ** -8
    lse = torch.full((1, 16, 1), 4.0, device="cuda")
    x = torch.einsum("hgd,hjd->hgj", q.float().view(H, 2, d), keys) / math.sqrt(d)
    want = torch.exp(x.double() - 4).sum(1)
    old = w[1, :, :1000].double()
    bsa.cache_weigh(c, q, lse, w, seqs=i32(1), fresh=10)
    old[:, 990:] = 0
    got = w[1, :, :1000].double()
    assert ((got - old - want).abs() <= 1e-3 * (want + old)).all()
    before = got.clone()
    kept = bsa.cache_evict(c, w, i32(600), seqs=i32(1), recent=10)[0, :, :600].long()
    order = torch.sort(before[:, :990], stable=True, dim=1, descending=True).indices[:, :590].sort(1).values
    assert torch.equal(kept[:, :590], order) and torch.equal(kept[:, 590:], torch.arange(990, 1000, device="cuda").expand(H, 10))
    assert torch.equal(w[1, :, :600].double(), before.gather(1, kept))
    head = torch.arange(H, device="cuda").view(H, 1)
    now = k.view(torch.uint8)[table[1, :3].long()].permute(1, 0, 2, 3).reshape(H, 768, d)[:, :600]
    assert torch.equal(now, own.permute(1, 0, 2, 3).reshape(H, 1024, d)[head, kept])
    assert lens.tolist() == [0, 600] and table[1].tolist() == [pages - 1, 3, pages - 7] + [-1] * 5
    assert bsa.cache_status(c) == (0, 0)


def test_graph_and_streams(bsa):
    m = filled("e4m3", [300, 200], 2, 16, 16, 64, seed=11)
    gen = torch.Generator().manual_seed(3)
    w0 = heavy(gen, 2, 2, 304).cuda()
    q = torch.randn(2, 4, 1, 64, generator=gen).to(torch.bfloat16).cuda()
    lse = torch.full((2, 4, 1), 6.0, device="cuda")

    def run(c, w, stream=None):
        bsa.cache_weigh(c, q, lse, w, stream=stream)
        return bsa.cache_evict(c, w, i32(90, 90) if stream is None else keep, sink=2, recent=8, kept=kept, stream=stream)

    keep = i32(90, 90)
    outs = []
    for how in ("plain", "stream", "graph"):
        c, w = upload(bsa, m), w0.clone()
        kept = torch.zeros(2, 2, 304, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        if how == "plain":
            run(c, w)
        elif how == "stream":
            s = torch.cuda.Stream()
            run(c, w, s)
            s.synchronize()
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                bsa.cache_weigh(c, q, lse, w)
                bsa.cache_evict(c, w, keep, sink=2, recent=8, kept=kept)
            g.replay()
        torch.cuda.synchronize()
        assert bsa.cache_status(c) == (0, 0)
        outs.append([t.clone() for t in (w, kept, c.lens, c.block_table, c.refs, c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale)])
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))


def test_refusals(bsa):
    c = bsa.cache_create(8, 2, 16, 64, 2, 4)
    w = torch.zeros(2, 2, 64, device="cuda")
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 4, 1, device="cuda")
    for bad in (lambda: bsa.cache_weigh(c, q[..., :32], lse, w), lambda: bsa.cache_weigh(c, q, lse[:1], w), lambda: bsa.cache_weigh(c, q, lse.half(), w),
                lambda: bsa.cache_weigh(c, q, lse, w[:1]), lambda: bsa.cache_weigh(c, q, lse, w.double()), lambda: bsa.cache_weigh(c, q, lse, w.cpu()),
                lambda: bsa.cache_weigh(c, q, lse, w[:, :, ::2]), lambda: bsa.cache_weigh(c, q.float(), lse, w), lambda: bsa.cache_weigh(c, q, lse, w, seqs=i32(0)),
                lambda: bsa.cache_weigh(c, q, lse, w, mask=torch.ones(2, 2, 1, dtype=torch.uint8, device="cuda"), bk=64),
                lambda: bsa.cache_evict(c, w[:, :1], i32(1, 1)), lambda: bsa.cache_evict(c, w, i32(1, 1).long()),
                lambda: bsa.cache_evict(c, w, i32(1, 1).cpu()), lambda: bsa.cache_evict(c, w, i32(1, 1), seqs=i32(0)),
                lambda: bsa.cache_evict(c, w, i32(1, 1), kept=i32(1)), lambda: bsa.cache_evict(c, w, i32(1, 1), kept=torch.zeros(2, 2, 4, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bsa.cache_weigh(c, q, lse, w, fresh=-1), lambda: bsa.cache_weigh(c, q[:, :3], lse[:, :3].contiguous(), w),
                lambda: bsa.cache_weigh(c, q, lse, w, mask=torch.ones(2, 4, 1, dtype=torch.uint8, device="cuda"), bk=48),
                lambda: bsa.cache_evict(c, w, i32(1, 1, 1)), lambda: bsa.cache_evict(c, w, i32(1, 1), sink=-1), lambda: bsa.cache_evict(c, w, i32(1, 1), recent=-1)):
        with pytest.raises(bsa.BsaError):
            bad()
    bsa.cache_weigh(c, q, lse, w)      # an empty cache
    bsa.cache_evict(c, w, i32(0, 5))
    assert bsa.cache_status(c) == (0, 0) and (w == 0).all()

@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,nq,causal,bk", [(1, 1, False, 0), (4, 1, False, 32), (3, 7, True, 0), (3, 7, True, 64), (8, 20, False, 0),
                                            (8, 20, True, 32), (40, 1, False, 64)])
def test_a_row_without_a_sum_gives_nothing_whatever_the_keys_are(bsa, kind, d, g, nq, causal, bk):
    """Keys and scales that are no numbers, seen by rows whose LSE is -inf alone."""
    gen = torch.Generator().manual_seed(g + d)
    m = filled(kind, [150, 75], 2, 64, 32, d, seed=8)
    q = (torch.randn(2, 2 * g, nq, d, generator=gen) * 0.2).to(torch.bfloat16).cuda()
    lse = torch.randn(2, 2 * g, nq, generator=gen) + 3
    lse[0, :g] = -math.inf       # the first head of sequence 0: no row has a sum
    lse[1, g] = -math.inf        # one query head of several, and (masked) the only one that selects key block 0
    mask = None
    if bk:
        mask = torch.ones(2, 2 * g, 150 // bk + 1, dtype=torch.uint8)
        mask[1, g + 1:, 0] = 0
    w0 = torch.rand(2, 2, 192, generator=gen)
    plain, got = w0.cuda(), w0.cuda()
    kw = dict(mask=None if mask is None else mask.cuda(), bk=bk, causal=causal, fresh=0)
    bsa.cache_weigh(upload(bsa, m), q, lse.cuda(), plain, **kw)
    if kind == "e4m3":
        m.codes[0][m.table[0, 0], 0, 20] = 0x7F          # NaN
    m.scales[0][m.table[0, 1], 0, 0] = math.inf
    m.scales[0][m.table[0, 2], 0, 0] = math.nan
    if bk:
        m.scales[0][m.table[1, 0], 1, 0] = math.nan      # tokens 0 .. 31
    bsa.cache_weigh(upload(bsa, m), q, lse.cuda(), got, **kw)
    assert plain.isfinite().all() and torch.equal(plain, got)
    assert torch.equal(got[0, 0].cpu(), w0[0, 0])


@pytest.mark.parametrize("kind,page,sb,sink", [("e4m3", 16, 16, 32), ("int8", 32, 16, 70), ("e4m3", 64, 32, 64)])
def test_shared_pages_of_sinks(bsa, kind, page, sb, sink):
    """Pages that hold the first `sink` tokens alone are not written: other sequences may hold them too (a prompt that
    all begin with), and their cuts agree with the model's."""
    m = filled(kind, [300, 280, 290], 2, page, sb, 64, seed=4, spare=10)
    whole = sink // page          # pages of sinks alone
    for s in (1, 2):
        for j in range(whole):
            m.refs[m.table[s, j]] -= 1
            m.table[s, j] = m.table[0, j]
            m.refs[m.table[0, j]] += 1
    c = upload(bsa, m)
    gen = torch.Generator().manual_seed(5)
    w = heavy(gen, 3, 2, m.table.shape[1] * page)
    w = evict_both(bsa, m, c, w, [150, 140, 200], sink=sink, recent=20)
    assert bsa.cache_status(c) == (0, 0) and m.refs.max() == 3
    # a page of which one token is no sink is written: left as it is
    t = w.clone()
    bsa.cache_evict(c, t, i32(100), sink=whole * page - 1)
    assert bsa.cache_status(c) == (-1, 0)
    assert_state(c, m)
    assert torch.equal(t, w)
    # a budget below the sinks: what is kept are the first and the recent ones; pages behind are given back
    k = whole * page
    evict_both(bsa, m, c, w.cpu(), [k + 3] * 3, sink=1 << 30, recent=3)
    assert bsa.cache_status(c) == (0, 0)
    bsa.cache_evict(c, w, i32(k), sink=1 << 30, recent=3)
    assert bsa.cache_status(c) == (-1, 0)  # (the last three move into the shared page)
    assert_state(c, m)


@pytest.mark.parametrize("kind,page,sb,d,lens,Hkv,g,nq,causal,bk,fresh", [
    ("e4m3", 64, 32, 128, [150, 33], 2, 8, 1, False, 0, 1),          # 8 rows: the last in registers
    ("e4m3", 64, 64, 128, [150, 40], 1, 9, 1, False, 0, 0),          # 9: the first from shared memory
    ("int8", 32, 16, 128, [131, 64], 2, 4, 5, True, 0, 5),           # 20
    ("e4m3", 16, 16, 128, [97, 300], 1, 16, 1, False, 0, 1),         # 16
    ("int8", 64, 64, 128, [200, 31], 1, 8, 4, True, 0, 1 << 30),     # 32
    ("e4m3", 64, 64, 128, [200, 31], 1, 11, 3, True, 0, 3),          # 33: tiles of 16 keys
    ("int8", 64, 16, 64, [150, 33], 2, 8, 1, False, 0, 1),
    ("e4m3", 32, 32, 64, [150, 70], 1, 9, 1, False, 0, 1),
    ("int8", 16, 16, 64, [260, 64], 2, 4, 8, True, 0, 8),            # 32
    ("e4m3", 64, 64, 64, [260, 65], 1, 3, 11, True, 0, 11),          # 33
    ("e4m3", 64, 32, 64, [500, 131], 2, 3, 3, True, 32, 3),          # masked, rows in shared memory: two blocks a tile
    ("int8", 64, 64, 64, [500, 131], 1, 4, 5, True, 64, 500),
    ("e4m3", 32, 16, 128, [500, 131], 2, 3, 3, True, 32, 3),
    ("int8", 64, 64, 128, [500, 131], 1, 16, 2, True, 64, 2),
    ("e4m3", 64, 64, 128, [500, 131], 1, 33, 1, False, 32, 1),       # more heads of a group than lanes, 33 rows
    ("int8", 64, 64, 64, [500, 131], 1, 32, 1, False, 32, 1)])
def test_weights_at_the_borders_of_the_kernels(bsa, kind, page, sb, d, lens, Hkv, g, nq, causal, bk, fresh):
    gen = torch.Generator().manual_seed(sum(lens) + d + g)
    m = filled(kind, lens, Hkv, page, sb, d, seed=6)
    for s in m.scales:
        s *= np.float32(0.25)
    c = upload(bsa, m)
    B = len(lens)
    q = (torch.randn(B, Hkv * g, nq, d, generator=gen) * 0.5).to(torch.float16 if page == 32 else torch.bfloat16)
    lse = torch.randn(B, Hkv * g, nq, generator=gen) + 3
    lse[0, -1, 0] = -math.inf
    w0 = torch.rand(B, Hkv, m.table.shape[1] * page, generator=gen)
    mask = None
    if bk:
        mask = (np.random.default_rng(2).random((B, Hkv * g, max(lens) // bk + 1)) < 0.2).astype(np.uint8) * 3
        mask[:, :, 0::4], mask[:, :, 1::4] = 0, 1    # of four blocks the first for no head, the second for all
    weigh_both(bsa, m, c, q, lse, w0, mask=mask, bk=bk, causal=causal, fresh=fresh)
    assert bsa.cache_status(c) == (0, 0)
