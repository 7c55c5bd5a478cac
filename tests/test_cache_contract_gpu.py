"""GPU tests of what the 8-bit cache promises beyond the plain path: pages that
were used before, lists that are the cache's own, tables and lengths that are
wrong, values and scales in masked places, long contexts."""
import numpy as np
import pytest
import torch

from oracle import cache as OC
from test_cache_gpu import KINDS, assert_close, filled, i32, keep_of, rand, upload

pytestmark = pytest.mark.gpu


def assert_state(c, m, what=""):
    """Every array of the cache, bit for bit (scales may be NaN)."""
    bits = lambda a: np.ascontiguousarray(a).view(np.uint8)
    for name, got, want in (("table", c.block_table, m.table), ("lens", c.lens, m.lens), ("refs", c.refs, m.refs),
                            ("k", c.k, m.codes[0]), ("v", c.v, m.codes[1]), ("k_scale", c.k_scale, m.scales[0]),
                            ("v_scale", c.v_scale, m.scales[1])):
        got = got.view(torch.uint8) if name in "kv" else got
        assert np.array_equal(bits(got.cpu().numpy()), bits(want)), (what, name)


def append_both(bsa, m, c, k, v, seqs, start, counts=None):
    m.append(k.double().numpy(), v.double().numpy(), seqs, counts, start)
    bsa.cache_append(c, k.cuda(), v.cuda(), seqs=i32(*seqs), start=i32(*start),
                     counts=None if counts is None else i32(*counts))


def assert_scales_of_their_tokens(c, seq, x, sb, kind, first=0):
    """Every block of the sequence (from token `first` on) has the scale that its tokens x [heads, n, d]
    need, and each value is off by two roundings at most: half a step each, 2^-4
    of the value (or half the scale's smallest step, 2^-10) for E4M3, half the
    scale for INT8."""
    page, n = c.page_size, x.shape[1]
    table = c.block_table[seq].tolist()
    codes = c.k.view(torch.uint8).cpu().numpy()
    for b0 in range(first, n, sb):
        p, r = table[b0 // page], b0 % page
        for h in range(x.shape[0]):
            new = x[h, b0:b0 + sb].double().numpy()
            sc = OC.scale_for(np.abs(new).max(), kind)
            assert float(c.k_scale[p, h, r // sb]) == sc, (b0, h)
            got = OC.decode(codes[p, h, r:r + new.shape[0]], kind) * sc
            step = np.maximum(np.abs(new) * 2.0 ** -4, sc * 2.0 ** -10) if kind == "e4m3" else 0.5 * sc
            assert (np.abs(got - new) <= 2.2 * step).all(), (b0, h)


# ------------------------------------------------------- pages used before

PIECES = [[(0, 100), (100, 28)], [(0, 32), (32, 32), (64, 64)], [(64, 64), (0, 64)], [(100, 28), (33, 67), (0, 33)]]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pieces", PIECES)
@pytest.mark.parametrize("page,sb,d", [(64, 64, 128), (32, 16, 64), (256, 128, 64)])
def test_room_filled_in_pieces_on_used_pages(bsa, kind, pieces, page, sb, d):
    m = OC.CacheModel(2 * 128 // page + 2, 2, page, d, 2, 8, kind, sb, seed=page)
    c = upload(bsa, m)
    g = torch.Generator().manual_seed(page)
    full = 2 * max(128, page)
    assert m.resize([full], [0]) == 0
    bsa.cache_resize(c, i32(full), i32(0))
    big = rand(g, 1, 2, full, d) * 2.0 ** 20
    append_both(bsa, m, c, big, big, [0], [0])
    m.resize([0], [0])
    bsa.cache_free(c, i32(0))
    assert m.resize([128], [1]) == 0
    bsa.cache_resize(c, i32(128), i32(1))
    assert_state(c, m, "handed out")
    x = rand(g, 1, 2, 128, d)
    for at, n in pieces:
        append_both(bsa, m, c, x[:, :, at:at + n], x[:, :, at:at + n], [1], [at])
        assert_state(c, m, f"piece {at}")
    assert_scales_of_their_tokens(c, 1, x[0], sb, kind)
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 0.0, 1e30])
def test_pools_that_were_never_written(bsa, kind, fill):
    page, sb, d = 32, 16, 64
    m = OC.CacheModel(8, 2, page, d, 2, 4, kind, sb, seed=3)
    for s in m.scales:
        s[:] = fill
    c = upload(bsa, m)
    g = torch.Generator().manual_seed(3)
    x = rand(g, 1, 2, 90, d)
    assert m.resize([90], [0]) == 0
    bsa.cache_resize(c, i32(90), i32(0))
    for at, n in ((0, 5), (5, 20), (60, 30), (25, 35)):
        append_both(bsa, m, c, x[:, :, at:at + n], x[:, :, at:at + n], [0], [at])
        assert_state(c, m, f"piece {at}")
    assert_scales_of_their_tokens(c, 0, x[0], sb, kind)
    # A step of one token at a time, into blocks whose scale nobody has written.
    y = rand(g, 40, 1, 2, 1, d)
    for i in range(30):
        assert m.resize([i + 1], [1]) == 0
        bsa.cache_resize(c, i32(i + 1), i32(1))
        append_both(bsa, m, c, y[i], y[i], [1], [i])
    assert_state(c, m, "steps")
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_held_tokens_of_no_scale(bsa, kind):
    """A table made by hand over memory that was never written: what lies in the
    block counts for nothing, the first tokens stored set its scale."""
    for fill in (float("nan"), float("inf"), -float("inf"), -2.0, 0.0):
        m = OC.CacheModel(3, 2, 64, 64, 1, 2, kind, 64, seed=5)
        m.table[0, :2], m.refs[:2], m.lens[0] = (1, 0), 1, 100
        for s in m.scales:
            s[:] = fill
        c = upload(bsa, m)
        x = rand(torch.Generator().manual_seed(5), 1, 2, 100, 64)
        for at, n in ((10, 20), (70, 3), (0, 64), (64, 36)):
            append_both(bsa, m, c, x[:, :, at:at + n], x[:, :, at:at + n], [0], [at])
            assert_state(c, m, f"{fill} {at}")
        assert_scales_of_their_tokens(c, 0, x[0], 64, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_past_a_shrunk_length(bsa, kind):
    """What a sequence (or one that shares its page) stored past its present
    length is no scale of what comes next; sharers keep theirs."""
    m = OC.CacheModel(12, 2, 64, 64, 3, 3, kind, 16, seed=7)
    c = upload(bsa, m)
    g = torch.Generator().manual_seed(7)

    def both(lens, seqs):
        assert m.resize(lens, seqs) == 0
        bsa.cache_resize(c, i32(*lens), i32(*seqs))
        assert_state(c, m, f"resize {lens} {seqs}")

    both([60], [0])
    big = rand(g, 1, 2, 60, 64) * 2.0 ** 20
    big[:, :, :20] *= 2.0 ** -20
    append_both(bsa, m, c, big, big, [0], [0])
    bsa.cache_fork(c, i32(0, 0), i32(1, 2))
    m.fork([0, 0], [1, 2])
    both([20, 33], [1, 2])
    # In one call: 0 takes a copy (with all its blocks), 2 takes one (three blocks),
    # 1 keeps the page; 1's and 2's other blocks begin anew, 0's stay.
    both([70, 64, 50], [0, 2, 1])
    x = rand(g, 1, 2, 60, 64)
    x[:, :, :20] = big[:, :, :20]
    append_both(bsa, m, c, x[:, :, 20:30], x[:, :, 20:30], [1], [20])
    append_both(bsa, m, c, x[:, :, 40:50], x[:, :, 40:50], [1], [40])
    append_both(bsa, m, c, x[:, :, 30:40], x[:, :, 30:40], [1], [30])
    assert_state(c, m)
    # (tokens 16 .. 19 were stored beside larger ones: that block's scale stays)
    assert_scales_of_their_tokens(c, 1, x[0, :, :50], 16, kind, 32)
    k = m.values(0)[0][:, 40:60]
    want = big[0, :, 40:60].double().numpy()
    assert np.abs(k - want).max() <= np.abs(want).max() * 2.0 ** -3
    # Alone with its page: shrunk and grown again.
    both([5], [2])
    both([64], [2])
    append_both(bsa, m, c, x[:, :, 16:26], x[:, :, 16:26], [2], [16])
    append_both(bsa, m, c, x[:, :, 26:32], x[:, :, 26:32], [2], [26])
    assert_state(c, m)
    p = int(m.table[2, 0])
    for h in range(2):
        sc = OC.scale_for(float(x[0, h, 16:32].abs().max()), kind)
        assert float(c.k_scale[p, h, 1]) == sc and float(c.v_scale[p, h, 1]) == sc
    assert bsa.cache_status(c) == (0, 0)


def test_scales_of_many_pages_and_copies(bsa):
    """Growth of many sequences over many pages with many scales each: all those
    of the pages taken are 0, all those of copied pages are the copied ones."""
    rng = np.random.default_rng(12)
    m = OC.CacheModel(3000, 3, 128, 64, 400, 12, "int8", 16, seed=12)
    lens = rng.integers(1, 300, 200).astype(np.int32)
    assert m.resize(lens) == 0
    m.fork(range(200), range(200, 400))
    for s in m.scales:
        s[:] = np.exp2(rng.integers(-9, 9, s.shape))
    c = upload(bsa, m)
    seqs = rng.permutation(400).astype(np.int32)
    want = np.concatenate([lens, lens])[seqs] + rng.integers(0, 500, 400).astype(np.int32)
    want = np.minimum(want, 12 * 128).astype(np.int32)
    bsa.cache_resize(c, torch.from_numpy(want).cuda(), torch.from_numpy(seqs).cuda())
    assert m.resize(want, seqs) == 0
    assert_state(c, m)
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_append_beside_tokens_of_the_largest_scales(bsa, kind):
    """Scales up to 2^127 are powers of two too (a cache filled by others)."""
    for e in (125, 126, 127):
        m = OC.CacheModel(2, 1, 16, 64, 1, 1, kind, 16, seed=9)
        assert m.resize([16]) == 0
        for s in m.scales:
            s[:] = 2.0 ** e
        for x in m.codes:
            x[:] = 0x08
        c = upload(bsa, m)
        x = rand(torch.Generator().manual_seed(e), 1, 1, 3, 64).clamp(-1.9, 1.9) * 2.0 ** 127
        append_both(bsa, m, c, x, x * 2.0 ** -3, [0], [7])
        assert OC.decode(m.codes[0][m.table[0, 0], 0, 7:10], kind).any()
        assert_state(c, m, f"2^{e}")


# ------------------------------------------- lists that are the cache's own

def test_lists_that_are_the_lengths_of_a_cache(bsa):
    """The lengths that a resize is still writing, as the counts of the append
    behind it and as the new lengths of another cache."""
    heads, page, d, n = 2, 16, 64, 700
    g = torch.Generator().manual_seed(13)
    rng = np.random.default_rng(13)
    c = bsa.cache_create(4 * n, heads, page, d, n, 4)
    other = bsa.cache_create(4 * n, heads, page, d, n, 4)
    x = rand(g, n, heads, 4 * page, d)
    xd = x.cuda()
    for turn in range(20):
        lens = torch.from_numpy(rng.integers(1, 4 * page + 1, n).astype(np.int32)).cuda()
        bsa.cache_free(c)
        bsa.cache_resize(c, lens)
        bsa.cache_append(c, xd, xd, counts=c.lens)
        bsa.cache_resize(other, c.lens)
        assert bsa.cache_status(c) == (0, 0) and bsa.cache_status(other) == (0, 0), turn
        assert torch.equal(c.lens, lens) and torch.equal(other.lens, lens), turn
        if turn % 10 == 9:
            m = OC.CacheModel(4 * n, heads, page, d, n, 4, seed=0)
            m.resize(lens.cpu().numpy())
            m.append(x.double().numpy(), x.double().numpy(), counts=lens.cpu().numpy())
            for s in range(0, n, 37):
                k = m.values(s)[0]
                p, L = c.block_table[s].cpu().numpy(), int(lens[s])
                got = np.concatenate([OC.decode(c.k[int(j)].view(torch.uint8).cpu().numpy(), "e4m3")
                                      * c.k_scale[int(j)].double().cpu().numpy().repeat(16, 1)[..., None]
                                      for j in p[:-(-L // page)]], 1)[:, :L]
                assert np.array_equal(got, k), s


# ------------------------------------- tables and lengths that are wrong

@pytest.mark.parametrize("kind,page,sb,d,nq", [("e4m3", 64, 32, 128, 1), ("int8", 16, 16, 64, 3), ("e4m3", 16, 16, 128, 5),
                                               ("int8", 256, 64, 128, 1), ("e4m3", 32, 16, 64, 30)])
@pytest.mark.parametrize("masked", [False, True])
def test_keys_of_no_page_are_not_attended(bsa, kind, page, sb, d, nq, masked):
    lens = [700, 700, 333, 2000]
    m, c = filled(bsa, lens, 2, page, sb, d, kind, -(-2000 // page), seed=17)
    c.k_scale.mul_(torch.where(torch.arange(c.num_pages, device="cuda") == 0, 4.0, 1.0).view(-1, 1, 1))
    m.scales[0] = c.k_scale.cpu().numpy()
    g = torch.Generator().manual_seed(17)
    q = rand(g, 4, 4, nq, d)
    mask = (torch.rand(4, 4, 2000 // 64, generator=g) < 0.7).to(torch.uint8) if masked else None
    good = bsa.cache_attention(c, q.cuda(), mask=None if mask is None else mask.cuda(), bk=64, causal=nq > 1)
    bad = {0: [0], 1: [-(-700 // page) - 1, 1], 3: range(0, -(-2000 // page), 2)}
    for s, js in bad.items():
        for i, j in enumerate(js):
            c.block_table[s, j] = (-1, c.num_pages, 1 << 30, -(1 << 31))[i % 4]
    o, lse = bsa.cache_attention(c, q.cuda(), mask=None if mask is None else mask.cuda(), bk=64, causal=nq > 1)
    st, det = bsa.cache_status(c)
    assert st == -7 and det in bad
    assert torch.equal(o[2], good[0][2]) and torch.equal(lse[2], good[1][2])
    for s in (0, 1, 3):
        k, v = m.values(s)
        keep = keep_of(k.shape[1], nq, 4, nq > 1, None if mask is None else mask[s].numpy(), 64)
        for j in bad[s]:
            keep[:, :, j * page:(j + 1) * page] = False
        assert_close(o[s], lse[s], OC.attention(q[s].double().numpy(), k, v, keep), q, k.shape[1], f"sequence {s}")
    c.block_table[3] = -1  # no page at all
    o, lse = bsa.cache_attention(c, q.cuda(), causal=nq > 1)
    assert not o[3].any() and torch.isneginf(lse[3]).all()
    assert bsa.cache_status(c)[0] == -7


def test_forward_of_a_sequence_with_no_page(bsa):
    m, c = filled(bsa, [600, 512, 600, 300], 2, 32, 32, 64, "e4m3", 20, seed=19)
    g = torch.Generator().manual_seed(19)
    p = bsa.plan(torch.ones(4, 4, 2, 8, dtype=torch.uint8, device="cuda"), 64, 64, 2)
    q = rand(g, 4, 4, 128, 64).cuda()
    good = bsa.cache_forward(p, c, q, causal=True)
    for s, j in ((1, 0), (2, 15)):
        was = int(c.block_table[s, j])
        for x in (-1, c.num_pages, 1 << 30):
            c.block_table[s, j] = x
            o, lse = bsa.cache_forward(p, c, q, causal=True)
            assert bsa.cache_status(c) == (-7, s) and bsa.sync_status(p)[0] == 0
            assert not o[s].any() and torch.isneginf(lse[s]).all()
            for b in {0, 1, 2, 3} - {s}:
                assert torch.equal(o[b], good[0][b]) and torch.equal(lse[b], good[1][b])
        c.block_table[s, j] = was
    c.block_table[2, 17] = -1  # past the plan's keys
    o, lse = bsa.cache_forward(p, c, q, causal=True)
    assert bsa.cache_status(c) == (0, 0)
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


def test_lengths_out_of_range_are_reported(bsa):
    m, c = filled(bsa, [600, 512, 300], 2, 32, 32, 64, "e4m3", 20, seed=23)
    g = torch.Generator().manual_seed(23)
    p = bsa.plan(torch.ones(3, 4, 2, 10, dtype=torch.uint8, device="cuda"), 64, 64, 2)
    q1, q2 = rand(g, 3, 4, 1, 64).cuda(), rand(g, 3, 4, 128, 64).cuda()
    mask = torch.ones(3, 4, 10, dtype=torch.uint8, device="cuda")
    calls = (lambda: bsa.cache_attention(c, q1), lambda: bsa.cache_attention(c, q1, mask=mask, bk=64),
             lambda: bsa.cache_forward(p, c, q2, causal=True))
    good = [f() for f in calls]
    assert bsa.cache_status(c) == (0, 0)
    for s, n in ((1, 641), (1, -1), (0, 2 ** 31 - 1), (2, -2 ** 31)):
        was = int(c.lens[s])
        c.lens[s] = n
        for f, want in zip(calls, good):
            o, lse = f()
            assert bsa.cache_status(c) == (-1, s), n
            assert not o[s].any() and torch.isneginf(lse[s]).all()
            for b in {0, 1, 2} - {s}:
                assert torch.equal(o[b], want[0][b]) and torch.equal(lse[b], want[1][b])
        c.lens[s] = was
    c.lens[1] = 640  # the most there is room for
    c.block_table[1] = c.block_table[0]
    bsa.cache_attention(c, q1)
    assert bsa.cache_status(c)[0] != -1


def test_page_operations_skip_sequences_of_bad_tables(bsa):
    for bad in (-1, 20, 1 << 30):
        m = OC.CacheModel(20, 1, 16, 64, 5, 6, seed=4)
        assert m.resize([60, 40, 20, 33]) == 0
        c = upload(bsa, m)

        def same(what, skip=None):
            t, w = c.block_table.cpu().numpy(), m.table.copy()
            if skip is not None:
                w[skip] = bad
            assert np.array_equal(t, w), (what, bad)
            assert np.array_equal(c.lens.cpu().numpy(), m.lens) and np.array_equal(c.refs.cpu().numpy(), m.refs), (what, bad)

        c.block_table[0, 2] = bad
        bsa.cache_resize(c, i32(20, 50), i32(0, 1))      # would give the bad page back
        assert m.resize([50], [1]) == 0
        assert bsa.cache_status(c) == (-7, 0)
        same("shrink", (0, 2))
        bsa.cache_fork(c, i32(0, 2), i32(4, 0))          # (0 is a source)
        assert bsa.cache_status(c)[0] == -1
        bsa.cache_fork(c, i32(0), i32(4))
        assert bsa.cache_status(c) == (-7, 0)
        same("fork", (0, 2))
        bsa.cache_resize(c, i32(49), i32(0))             # the bad page stays
        m.resize([49], [0])
        assert bsa.cache_status(c) == (0, 0)
        same("shrink behind it", (0, 2))
        c.block_table[0, 2] = int(m.table[0, 2])
        c.block_table[3, 2] = bad                        # its partly filled last page
        bsa.cache_resize(c, i32(34, 21), i32(3, 2))
        assert m.resize([21], [2]) == 0
        assert bsa.cache_status(c) == (-7, 3)
        same("grow", (3, 2))
        # Freed, by either call, a sequence gives back what pages it has.
        bsa.cache_resize(c, i32(0), i32(3))
        assert bsa.cache_status(c) == (-7, 3)
        held = m.table[3, 2]
        m.resize([0], [3])
        m.refs[held] = 1
        same("free")
        c.refs[int(held)] = 0
        m.refs[held] = 0
        c.block_table[1, 1] = bad
        bsa.cache_free(c, i32(1))
        assert bsa.cache_status(c) == (-7, 1)
        held = m.table[1, 1]
        m.resize([0], [1])
        m.refs[held] = 1
        same("free of a list")


# -------------------------------------------------- small weights, long rows

@pytest.mark.parametrize("kind,d", [("int8", 64), ("e4m3", 128)])
@pytest.mark.parametrize("octaves", [25.05, 28.0, 30.0])
def test_a_long_tail_below_a_sink(bsa, kind, d, octaves):
    """Keys ahead that outweigh every other one 2^octaves times, then a flat
    tail, long enough to count.  A weight is off by half of fp16's least step at
    2^7 times the row's reference, 2^-32 of that, so the tail's part by n 2^-32;
    the scores by what assert_close derives; and half a step of bf16."""
    n, B = 1 << 17, 320  # (rows enough that a piece of the work is a whole row)
    tile = 4096 // d
    c = bsa.cache_create(n // 256, 1, 256, d, 1, n // 256, kind, 256)
    c.block_table[0] = torch.arange(n // 256, dtype=torch.int32)
    c.refs.fill_(1)
    c.lens[0] = n
    one = {"int8": 1, "e4m3": 0x38}[kind]
    sinks = torch.arange(4) * tile                       # one for each warp
    k, v = (x.view(torch.uint8).view(-1, d) for x in (c.k, c.v))
    k[sinks, 0] = one
    v.fill_(one)
    v[sinks] = 0
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    q = torch.zeros(B, 1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = octaves * float(np.log(2.0))
    o, lse = bsa.cache_attention(c, q, seqs=torch.zeros(B, dtype=torch.int32, device="cuda"), scale=scale)
    tail = (n - 4) * 2.0 ** -octaves
    want = tail / (4 + tail)
    bound = want * (2.0 ** -8 + 4 * scale * 2.0 ** -23 + 2.0 ** -11) + n * 2.0 ** -32 / (4 + tail) + 2.0 ** -25
    assert bound < want / 2
    err = (o.double() - want).abs().max().item()
    assert err <= bound, (err / bound, err / want)
    # A thread sums n / 32 of a row's weights (4 warps, 8 threads to a row); where
    # the sink is its first, each addition is off by half a unit of fp32's last
    # place, 2^-24 of the sum.
    lse_bound = n / 32 * 2.0 ** -24 + 1e-5
    assert (lse.double() - (scale + np.log(4 + tail))).abs().max().item() <= lse_bound
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("kind,d", [("int8", 64), ("e4m3", 128)])
@pytest.mark.parametrize("nq", [1, 20])
def test_long_flat_rows(bsa, kind, d, nq):
    """Rows whose keys all weigh about the same, with a bound that an output of
    zeros fails: weights lose 2^-11 of themselves (they are far above 2^-14 of
    the reference), so O half a step and 2^-11 of the mean of |v|."""
    n = 30000
    m, c = filled(bsa, [n, 777], 2, 64, 64, d, kind, -(-n // 64), seed=41)
    g = torch.Generator().manual_seed(41)
    q = rand(g, 2, 4, nq, d) * 2.0 ** -4
    o, lse = bsa.cache_attention(c, q.cuda(), causal=nq > 1)
    for b in range(2):
        k, v = m.values(b)
        O, L, A, mag = OC.attention(q[b].double().numpy(), k, v, keep_of(k.shape[1], nq, 4, nq > 1))
        ds = mag * (d + 4) * 2.0 ** -23 + 2.0 ** -21
        bound = 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2 * ds[..., None]) * 2 * A
        assert b == 1 or np.median(bound / np.abs(O)) < 0.5
        err = np.abs(o[b].double().cpu().numpy() - O)
        assert (err <= bound).all(), float((err / bound).max())
        assert (np.abs(lse[b].double().cpu().numpy() - L) <= ds + k.shape[1] * 2.0 ** -24 + 1e-5).all()


# --------------------------------------------- scales in places not attended

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,sb", [(64, 16), (64, 64), (128, 16), (128, 32)])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_scales_of_blocks_that_a_row_does_not_attend(bsa, kind, d, sb, fill):
    """The scales of a block reach only the rows that attend a key of it: rows
    cut off by causality or by a mask of blocks, beside rows that are not."""
    lens = [200, 128 + sb]
    m, c = filled(bsa, lens, 1, 64, sb, d, kind, 4, seed=47)
    g = torch.Generator().manual_seed(47)

    def spoil(seq, key):
        p = int(m.table[seq, key // 64])
        c.v_scale[p, :, key % 64 // sb] = fill
        return p

    # Causal: the last sb keys in a block of their own, seen by the last queries only.
    q = rand(g, 1, 2, sb + 4, d)
    spoil(1, 128)
    o, lse = bsa.cache_attention(c, q.cuda(), seqs=i32(1), causal=True)
    assert torch.isfinite(o[:, :, :4]).all() and not torch.isfinite(o[:, :, 4:]).any()
    k, v = m.values(1)
    ref = OC.attention(q[0].double().numpy(), k, v, keep_of(128 + sb, sb + 4, 2, True))
    assert_close(o[0, :, :4], lse[0, :, :4], [x[:, :4] for x in ref], q, 128 + sb, "causal")
    # A mask of 32 keys: head 0 leaves out what head 1 attends.
    if sb <= 32:
        q = rand(g, 1, 2, 1, d)
        spoil(0, 32)
        mask = torch.ones(1, 2, 7, dtype=torch.uint8)
        mask[0, 0, 1] = 0
        o, lse = bsa.cache_attention(c, q.cuda(), seqs=i32(0), mask=mask.cuda(), bk=32)
        assert torch.isfinite(o[0, 0]).all() and not torch.isfinite(o[0, 1]).any()
        k, v = m.values(0)
        ref = OC.attention(q[0].double().numpy(), k, v, keep_of(200, 1, 2, False, mask[0].numpy(), 32))
        assert_close(o[0, :1], lse[0, :1], [x[:1] for x in ref], q, 200, "mask")
        # Nobody attends it: nobody sees it.
        mask[0, 1, 1] = 0
        o, lse = bsa.cache_attention(c, q.cuda(), seqs=i32(0), mask=mask.cuda(), bk=32)
        ref = OC.attention(q[0].double().numpy(), k, v, keep_of(200, 1, 2, False, mask[0].numpy(), 32))
        assert_close(o[0], lse[0], ref, q, 200, "nobody")
    assert bsa.cache_status(c) == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_queries_down_to_the_least_numbers(bsa, d):
    """Rows of q below 2^-100 with a scale to match keep their bits."""
    m, c = filled(bsa, [300, 90], 1, 32, 32, d, "int8", 10, seed=53)
    g = torch.Generator().manual_seed(53)
    for e in (-105, -114, -119):
        q = rand(g, 2, 4, 1, d) * 2.0 ** e
        scale = 2.0 ** (-e - 3)
        o, lse = bsa.cache_attention(c, q.cuda(), scale=scale)
        for b in range(2):
            k, v = m.values(b)
            ref = OC.attention(q[b].double().numpy(), k, v, keep_of(k.shape[1], 1, 4), scale)
            assert_close(o[b], lse[b], ref, q, k.shape[1], f"2^{e}")


def test_two_threads_resize_caches_by_long_lists(bsa):
    """Lists whose sizes need different amounts of shared memory, at once."""
    import threading
    caches = [bsa.cache_create(16, 1, 16, 64, 4096, 1) for _ in range(2)]
    lists = [torch.full((n,), 0, dtype=torch.int32, device="cuda") for n in (4096, 3500)]
    torch.cuda.synchronize()
    bad = []
    start = threading.Barrier(2)

    def work(i):
        stream = torch.cuda.Stream()
        try:
            start.wait()
            for _ in range(1000):
                bsa.cache_resize(caches[i], lists[i], stream=stream)
        except Exception as e:
            bad.append(repr(e))
        torch.cuda.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    assert all(bsa.cache_status(c) == (0, 0) for c in caches)


def test_a_context_of_the_callers_own_stays_current(bsa):
    """A thread that works in a context made with the driver's API: its first
    call runs there, and leaves it current."""
    import ctypes
    import threading
    from block_sparse_attention_plan_gb300 import _cache
    lib, cu = _cache._library(), ctypes.CDLL("libcuda.so.1")
    out = {}

    def work():
        ctx, now, at = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_uint64()
        ok = [cu.cuInit(0), cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0), cu.cuMemAlloc_v2(ctypes.byref(at), 4096)]
        if any(ok):
            out["skip"] = ok
            return
        f = lambda o: ctypes.c_void_p(at.value + o)
        c = _cache.CacheC(f(0), f(0), f(0), f(0), f(256), f(512), f(768), f(1024), 0, 8, 1, 16, 64, 16, 4, 4)
        out["status"] = lib.bsa_cache_init(ctypes.byref(c), None)
        cu.cuCtxGetCurrent(ctypes.byref(now))
        out["same"] = now.value == ctx.value
        table = (ctypes.c_int32 * 16)()
        out["copied"] = cu.cuMemcpyDtoH_v2(table, ctypes.c_uint64(at.value + 256), 64)
        out["table"] = list(table)
        cu.cuMemFree_v2(at)
        cu.cuCtxDestroy_v2(ctx)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if "skip" in out:
        pytest.skip(f"no context: {out['skip']}")
    assert out == {"status": 0, "same": True, "copied": 0, "table": [-1] * 16}


# ------------------------------------------------- forms that no test above has

@pytest.mark.parametrize("kind,page,sb,d,g,nq,bk", [
    ("int8", 16, 16, 64, 4, 1, 32), ("e4m3", 32, 32, 64, 8, 1, 64), ("int8", 32, 16, 64, 2, 13, 128),
    ("int8", 64, 64, 128, 4, 30, 32), ("e4m3", 16, 16, 64, 7, 20, 32), ("e4m3", 128, 64, 64, 2, 60, 256),
    ("int8", 256, 256, 128, 1, 5, 64)])
def test_block_masks_of_every_form(bsa, kind, page, sb, d, g, nq, bk):
    """Masks in values: tiles over two mask blocks (d 64), both code types, small
    pages, more than 96 rows; the mask ends before the longest sequence, at an
    odd number of blocks."""
    lens = [1000, 130, 641, 1, 0, 33]
    m, c = filled(bsa, lens, 2, page, sb, d, kind, -(-1000 // page), seed=bk + nq)
    gen = torch.Generator().manual_seed(bk + nq)
    mask = (torch.rand(6, 2 * g, 960 // bk | 1, generator=gen) < 0.4).to(torch.uint8) * 5
    mask[0, 0], mask[2, g:] = 0, 0
    q = rand(gen, 6, 2 * g, nq, d)
    for causal in (False, True):
        o, lse = bsa.cache_attention(c, q.cuda(), mask=mask.cuda(), bk=bk, causal=causal)
        assert bsa.cache_status(c) == (0, 0)
        for b, n in enumerate(lens):
            k, v = m.values(b)
            ref = OC.attention(q[b].double().numpy(), k, v, keep_of(n, nq, 2 * g, causal, mask[b].numpy(), bk))
            assert_close(o[b], lse[b], ref, q, n, f"row {b} causal {causal}")


def test_forward_with_split_weights(bsa):
    m, c = filled(bsa, [400, 256], 2, 64, 64, 128, "e4m3", 8, seed=61)
    g = torch.Generator().manual_seed(61)
    mask = (torch.rand(2, 4, 2, 4, generator=g) < 0.8).to(torch.uint8)
    mask[:, :, :, 0] = 1
    p = bsa.plan(mask.cuda(), 64, 128, 2)
    q = rand(g, 2, 4, 128, 128)
    o, lse = bsa.cache_forward(p, c, q.cuda(), causal=True, split=True)
    assert bsa.sync_status(p)[0] == 0 and bsa.cache_status(c) == (0, 0)
    from compare import assert_attention_close
    refs = []
    for b in range(2):
        k, v = m.values(b)
        keep = keep_of(k.shape[1], 128, 4, True)
        keep &= mask[b].numpy().astype(bool).repeat(64, 1).repeat(128, 2)[:, :, :k.shape[1]]
        refs.append(OC.attention(q[b].double().numpy(), k, v, keep)[:2])
    assert_attention_close(o, lse, np.stack([r[0] for r in refs]), np.stack([r[1] for r in refs]), "split")


def test_too_few_pages_take_the_releases_back(bsa):
    """A list that gives pages back (shared ones too) and still lacks some
    changes nothing at all."""
    m = OC.CacheModel(10, 2, 16, 64, 5, 6, "e4m3", 16, seed=4)
    assert m.resize([60, 40, 20]) == 0
    m.fork([0], [3])
    c = upload(bsa, m)
    for lens, seqs in (([16, 0, 96, 70], [0, 1, 2, 3]), ([0, 96, 96], [3, 1, 2]), ([0, 0, 96, 96], [0, 1, 2, 4])):
        before = m.refs.copy()
        missing = m.resize(lens, seqs)
        assert missing > 0 and np.array_equal(m.refs, before)
        bsa.cache_resize(c, i32(*lens), i32(*seqs))
        assert bsa.cache_status(c) == (-5, missing)
        assert_state(c, m, f"{lens} {seqs}")
    assert m.resize([16, 0, 50], [0, 1, 2]) == 0
    bsa.cache_resize(c, i32(16, 0, 50), i32(0, 1, 2))
    assert_state(c, m)


@pytest.mark.parametrize("kind,page,sb", [("e4m3", 32, 16), ("int8", 64, 16), ("int8", 16, 16)])
def test_page_operations_and_tokens_in_a_small_pool(bsa, kind, page, sb):
    """A seeded run of every operation in a pool that is often too small."""
    rng = np.random.default_rng(page + sb)
    gen = torch.Generator().manual_seed(page + sb)
    m = OC.CacheModel(24, 2, page, 64, 8, 7, kind, sb, seed=2)
    c = upload(bsa, m)
    refused = 0
    for step in range(150):
        op = int(rng.integers(6))
        live, empty = np.nonzero(m.lens)[0], np.nonzero(m.lens == 0)[0]
        if op <= 1:
            n = int(rng.integers(1, 6))
            seqs = rng.choice(8, n, replace=False)
            lens = m.lens[seqs] + rng.integers(0, 3, n) if op else rng.integers(0, 7 * page + 1, n)
            lens = np.minimum(lens, 7 * page)
            missing = m.resize(lens, seqs)
            bsa.cache_resize(c, i32(*lens.tolist()), i32(*seqs.tolist()))
            assert bsa.cache_status(c) == ((-5, missing) if missing else (0, 0)), step
            refused += missing > 0
        elif op == 2 and len(live) and len(empty):
            n = int(rng.integers(1, len(empty) + 1))
            src, dst = rng.choice(live, n).tolist(), rng.choice(empty, n, replace=False).tolist()
            m.fork(src, dst)
            bsa.cache_fork(c, i32(*src), i32(*dst))
        elif op == 3:
            m.compact()
            bsa.cache_compact(c)
        elif op == 4:
            s = int(rng.integers(8))
            m.resize([0], [s])
            bsa.cache_free(c, i32(s))
        elif len(live):
            s = int(rng.choice(live))
            n = int(rng.integers(1, m.lens[s] + 1))
            at = int(rng.integers(0, m.lens[s] - n + 1))
            x = rand(gen, 1, 2, n, 64) * 2.0 ** float(rng.integers(-8, 8))
            append_both(bsa, m, c, x, -x, [s], [at])
            bsa.cache_status(c)  # (tokens for shared pages are refused)
        assert_state(c, m, f"step {step} op {op}")
    assert refused >= 5


def test_tokens_and_queries_of_fp16(bsa):
    m = OC.CacheModel(8, 2, 32, 64, 2, 4, "e4m3", 16, seed=8)
    assert m.resize([100, 31]) == 0
    c = upload(bsa, m)
    g = torch.Generator().manual_seed(8)
    x = rand(g, 2, 2, 100, 64, dtype=torch.float16)
    append_both(bsa, m, c, x, x, [0, 1], [0, 0], [100, 31])
    assert_state(c, m)
    q = rand(g, 2, 8, 2, 64, dtype=torch.float16)
    o, lse = bsa.cache_attention(c, q.cuda(), causal=True)
    assert o.dtype == torch.float16
    for b, n in enumerate((100, 31)):
        k, v = m.values(b)
        assert_close(o[b], lse[b], OC.attention(q[b].double().numpy(), k, v, keep_of(n, 2, 8, True)), q, n, f"row {b}")
