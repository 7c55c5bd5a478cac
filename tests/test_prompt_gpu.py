"""GPU tests of the attention of packed prompts (bsa_prompt_attention) against fp64,
with bounds from the arithmetic."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import prompt as OP

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def ptr(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32)


def bounds(O, L, A, mag, dtype, n, vmax):
    """What rounding can do to O and LSE.  Scores: fp32 sums of d <= 128 exact products, within 128 2^-23 of
    sum |q k| (mag), and the product with scale log2(e), its difference with the reference and ex2, 2^-22 of terms
    of mag each.  A weight is off by that relatively and by half a step of the type (fp16 weights that leave its range,
    2^-32 of the row's largest), so O by as much of sum w |v| (A) and, normalised, once more by the scores' part;
    then O is rounded."""
    half = torch.finfo(dtype).eps / 2
    s = np.expm1(mag * (2.0 ** -16 + 2.0 ** -21) + 2.0 ** -20)
    tiny = n * 2.0 ** -31 * vmax if dtype == torch.float16 else 0.0
    return A * (half + 2 * s[..., None]) + (np.abs(O) + A * half) * half + tiny + 2.0 ** -24, s + 2.0 ** -21 * (1 + np.abs(L))


def check(bsa, q, k, v, offsets, causal=True, scale=None, **kw):
    """Runs on the GPU; q, k, v are CPU tensors (any strides)."""
    off = offsets.numpy()
    o, lse = bsa.prompt_attention(q.cuda(), k.cuda(), v.cuda(), offsets.cuda(), causal=causal, scale=scale, **kw)
    O, L, A, mag = OP.attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), off, causal, scale)
    rows = slice(off[0], off[-1])
    to, tl = bounds(O[rows], L[rows], A[rows], mag[rows], q.dtype, int(np.diff(off).max()), float(v.abs().max()))
    eo = np.abs(o.double().cpu().numpy()[rows] - O[rows])
    el = np.abs(lse.double().cpu().numpy()[rows] - L[rows])
    assert (eo <= to).all(), (np.nanmax(eo / to), np.argwhere(~(eo <= to))[:3])
    assert (el <= tl).all(), (np.nanmax(el / tl), np.argwhere(~(el <= tl))[:3])
    return o, lse


def rows(gen, T, H, d, dtype, amp=1.0):
    return (torch.randn(T, H, d, generator=gen) * amp).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [
    ([1], 1, 1, 64), ([0, 1, 0, 2, 3], 4, 1, 128), ([5, 64, 63, 65, 1], 8, 2, 128), ([127, 128, 129], 2, 2, 64),
    ([300, 7], 3, 1, 128), ([255, 257], 14, 2, 64), ([40, 0, 500], 16, 1, 64), ([33, 200], 32, 1, 128),
    ([700], 6, 3, 128), ([511, 513], 2, 1, 64)])
def test_against_the_oracle(bsa, dtype, causal, lens, Hq, Hkv, d):
    gen = torch.Generator().manual_seed(sum(lens) + Hq)
    T = sum(lens)
    check(bsa, rows(gen, T, Hq, d, dtype), rows(gen, T, Hkv, d, dtype), rows(gen, T, Hkv, d, dtype), ptr(lens), causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 4, 1), (64, 7, 1), (128, 2, 2)])
def test_long_prompts(bsa, dtype, d, Hq, Hkv):
    """Several blocks and items per CTA; references that move (scores grow along the keys), against torch in fp64."""
    gen = torch.Generator("cuda").manual_seed(d)
    lens = [3001, 1, 2177, 640]
    T = sum(lens)
    q, k, v = (torch.randn(T, h, d, device="cuda", generator=gen) for h in (Hq, Hkv, Hkv))
    k = k * torch.linspace(0.1, 4.0, T, device="cuda").view(-1, 1, 1)
    q, k, v = (x.to(dtype) for x in (q, k, v))
    off = ptr(lens)
    for causal in (True, False):
        o, lse = bsa.prompt_attention(q, k, v, off.cuda(), causal=causal)
        for a, b in zip(off.tolist(), off.tolist()[1:]):
            for h in range(Hq):
                qq, kk, vv = q[a:b, h].double(), k[a:b, h * Hkv // Hq].double(), v[a:b, h * Hkv // Hq].double()
                s = qq @ kk.T / math.sqrt(d)
                mag = (qq.abs() @ kk.abs().T / math.sqrt(d))
                if causal:
                    drop = torch.ones_like(s, dtype=torch.bool).triu_(1)
                    s, mag = s.masked_fill(drop, -math.inf), mag.masked_fill(drop, 0)
                w = torch.softmax(s, 1)
                to, tl = bounds((w @ vv).cpu().numpy(), torch.logsumexp(s, 1).cpu().numpy(), (w @ vv.abs()).cpu().numpy(),
                                mag.amax(1).cpu().numpy(), dtype, b - a, float(vv.abs().max()))
                eo = (o[a:b, h].double() - w @ vv).abs().cpu().numpy()
                el = (lse[a:b, h].double() - torch.logsumexp(s, 1)).abs().cpu().numpy()
                assert (eo <= to).all() and (el <= tl).all(), (a, h, (eo / to).max(), (el / tl).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,d,lens", [(1, 1, 128, [6677, 6570, 6463, 6636]), (1, 1, 64, [5001, 4000]), (4, 1, 128, [3000] * 3),
                                           (2, 2, 128, [129, 130, 128, 127, 1] * 20), (3, 1, 128, [20] * 40)])
def test_cold_and_warm_inputs(bsa, dtype, Hq, Hkv, d, lens):
    """Keys and values that come from memory, later ones now and then before earlier ones, and from L2: the same bits,
    and no wait that runs out."""
    T = sum(lens)
    off = ptr(lens).cuda()
    flush = torch.empty(400 << 20, dtype=torch.uint8, device="cuda")
    ws = torch.empty(bsa.prompt_workspace_bytes(len(lens), T, Hq, Hkv), dtype=torch.uint8, device="cuda")
    for seed in range(6):
        gen = torch.Generator("cuda").manual_seed(seed)
        q, k, v = (torch.randn(T, h, d, device="cuda", generator=gen).to(dtype) for h in (Hq, Hkv, Hkv))
        flush.fill_(seed)
        a = bsa.prompt_attention(q, k, v, off, causal=seed != 3, workspace=ws)
        assert bsa.prompt_status(ws) == (0, 0)
        b = bsa.prompt_attention(q, k, v, off, causal=seed != 3, workspace=ws)
        assert bsa.prompt_status(ws) == (0, 0)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[0].float()).all()


def test_many_prompts(bsa):
    """More prompts than a pass of the schedule takes, most of them empty or short."""
    rng = np.random.default_rng(0)
    lens = np.where(rng.random(2500) < 0.5, 0, rng.integers(1, 5, 2500))
    lens[1777] = 400
    gen = torch.Generator().manual_seed(0)
    T = int(lens.sum())
    check(bsa, rows(gen, T, 2, 64, torch.bfloat16), rows(gen, T, 1, 64, torch.bfloat16), rows(gen, T, 1, 64, torch.bfloat16), ptr(lens))


def test_rows_of_no_prompt_are_left(bsa):
    gen = torch.Generator().manual_seed(1)
    q, k, v = (rows(gen, 400, h, 128, torch.bfloat16) for h in (4, 2, 2))
    for x in (q, k, v):
        x[:37], x[37 + 300:] = math.nan, math.inf
    off = ptr([170, 0, 130], first=37)
    out = torch.full((400, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((400, 4), 6.0, device="cuda")
    check(bsa, q, k, v, off, out=out, lse=lse)
    assert (out[:37] == 5).all() and (out[337:] == 5).all() and (lse[:37] == 6).all() and (lse[337:] == 6).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,g", [(128, 4), (64, 1), (128, 32)])
def test_infinities_and_nan_stay_with_the_rows_that_attend_them(bsa, dtype, causal, d, g):
    gen = torch.Generator().manual_seed(2)
    lens = [150, 90, 300]
    T, H = sum(lens), 2 * g
    q, k, v = (rows(gen, T, h, d, dtype) for h in (H, 2, 2))
    clean = [x.clone() for x in (q, k, v)]
    v[20, 0, 3], v[149, 0, 5], v[150, 1, 0] = math.inf, math.nan, -math.inf      # prompt 0's last row, prompt 1's first
    v[260, 0, 7], v[500, 0, 7], v[539, 1, d - 1] = math.inf, -math.inf, math.nan  # both infinities in one column
    k[240 + 200, 1, 4] = math.nan
    k[130, 0, 4] = math.inf
    q[10, 0, 0] = math.nan
    off = ptr(lens)
    o, lse = bsa.prompt_attention(q.cuda(), k.cuda(), v.cuda(), off.cuda(), causal=causal)
    po, pl = bsa.prompt_attention(*(x.cuda() for x in clean), off.cuda(), causal=causal)
    o, lse, po, pl = (x.float().cpu() for x in (o, lse, po, pl))
    for b, (a, e) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        for h in range(H):
            kv = h // g
            for t in range(a, e):
                see = slice(a, t + 1 if causal else e)
                row_bad = bool(torch.isnan(q[t, h]).any() or torch.isnan(k[see, kv]).any())
                # an infinite key: the score is +inf (NaN), -inf (weight 0) or NaN
                s = (q[t, h].float() @ k[see, kv].float().T)
                if torch.isnan(s).any() or (s == math.inf).any():
                    row_bad = True
                if row_bad:
                    assert torch.isnan(o[t, h]).all() and torch.isnan(lse[t, h]), (t, h)
                    continue
                vv = v[see, kv].float()
                want = torch.where(torch.isfinite(vv), 0.0, vv).sum(0)   # inf + -inf is NaN
                fine = want == 0
                assert torch.isfinite(o[t, h][fine]).all(), (t, h)
                got = o[t, h][~fine]
                # (in a block that all rows attend as a whole the matrix product decides: an infinity whose weight is 0
                # there is NaN)
                assert (~torch.isfinite(got)).all(), (t, h)
                if not (s == -math.inf).any():
                    assert torch.equal(o[t, h][fine], po[t, h][fine]) and lse[t, h] == pl[t, h], (t, h)


def test_strides_and_given_outputs(bsa):
    gen = torch.Generator().manual_seed(3)
    T = 333
    qkv = rows(gen, T, 12, 128, torch.float16).cuda()              # one projection's heads: 8 q, 2 k, 2 v
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    off = ptr([133, 200]).cuda()
    want, wl = bsa.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), off)
    got, gl = bsa.prompt_attention(q, k, v, off)
    assert torch.equal(want, got) and torch.equal(wl, gl)
    # heads ahead of tokens; an output with 16-byte alignment only; no LSE wanted through the C ABI is another test
    hq = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    room = torch.zeros(T * 8 * 136 + 8, dtype=torch.float16, device="cuda")
    out = room[8:].view(T, 8, 136)[..., :128]
    got, gl = bsa.prompt_attention(*hq, off, out=out)
    assert got is out and torch.equal(want, out) and torch.equal(wl, gl)
    assert (room[8:].view(T, 8, 136)[..., 128:] == 0).all()
    # one head, one token: dimensions without a stride
    x = torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16)
    o, lse = bsa.prompt_attention(x.as_strided((1, 1, 64), (3, 5, 1)), x, x, ptr([1]).cuda())
    assert torch.equal(o, x)


def test_scale_and_large_scores(bsa):
    gen = torch.Generator().manual_seed(4)
    q, k, v = (rows(gen, 260, h, 64, torch.bfloat16, 6.0) for h in (2, 1, 1))
    check(bsa, q, k, v, ptr([260]), scale=0.5)
    check(bsa, q, k, v, ptr([260]), scale=1e-3, causal=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1500, 130, 700], [100, 1300], [40] * 3 + [2100]])
def test_references_that_move(bsa, dtype, d, lens):
    """Scores that rise by 30 or more a block, fall, or jump: the reference moves in every block of some rows, in
    none of others, in both tiles of an item and where an item has one."""
    gen = torch.Generator().manual_seed(d + len(lens))
    T = sum(lens)
    u = torch.randint(0, 2, (d,), generator=gen).double() * 2 - 1
    j = torch.arange(T).double()
    f = torch.stack([j / T * 40, 40 - j / T * 40, (j // 200 % 2) * 30], 1)  # a K/V head each
    k = (f[:, :, None] * u).to(dtype)
    q = ((torch.rand(T, 6, 1, generator=gen).double() + 0.25) * u).to(dtype)
    v = rows(gen, T, 3, d, dtype)
    check(bsa, q, k, v, ptr(lens))
    check(bsa, q, k, v, ptr(lens), causal=False)


def test_equal_keys_give_the_mean(bsa):
    v = torch.randn(500, 1, 128, generator=torch.Generator().manual_seed(5)).to(torch.float16)
    k = torch.ones(500, 1, 128, dtype=torch.float16)
    o, lse = bsa.prompt_attention(k.cuda(), k.cuda(), v.cuda(), ptr([500]).cuda())
    n = torch.arange(1, 501, dtype=torch.float64).view(-1, 1)
    mean = v[:, 0].double().cumsum(0) / n
    assert ((o[:, 0].double().cpu() - mean).abs() <= mean.abs() * 2.0 ** -11 + 2.0 ** -18).all()  # weights are equal and exact
    assert ((lse[:, 0].double().cpu() - (math.sqrt(128) + torch.log(n[:, 0]))).abs() <= 2.0 ** -18).all()


def test_bad_offsets_write_nothing(bsa):
    x = torch.randn(64, 2, 64, device="cuda").to(torch.bfloat16)
    ws = torch.empty(bsa.prompt_workspace_bytes(3, 64, 2, 2), dtype=torch.uint8, device="cuda")
    for bad in ([0, 30, 20, 64], [-1, 30, 40, 64], [0, 30, 40, 65], [0, 70, 10, 20]):
        out, lse = torch.full_like(x, 3.0), torch.full((64, 2), 3.0, device="cuda")
        bsa.prompt_attention(x, x, x, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out, lse=lse, workspace=ws)
        assert bsa.prompt_status(ws)[0] == -1 and (out == 3).all() and (lse == 3).all(), bad
    bsa.prompt_attention(x, x, x, torch.tensor([0, 30, 30, 64], dtype=torch.int32, device="cuda"), out=out, lse=lse, workspace=ws)
    assert bsa.prompt_status(ws) == (0, 0) and not (out == 3).all(2).any()  # (a single value may be 3)


def test_graph_streams_and_calls_in_a_row(bsa):
    gen = torch.Generator().manual_seed(6)
    q, k, v = (rows(gen, 1000, h, 128, torch.bfloat16).cuda() for h in (8, 2, 2))
    off = ptr([400, 3, 597]).cuda()
    want = [t.clone() for t in bsa.prompt_attention(q, k, v, off)]
    for _ in range(20):  # the same bits, calls queued up behind one another
        got = bsa.prompt_attention(q, k, v, off)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = bsa.prompt_attention(q, k, v, off, stream=s), bsa.prompt_attention(q, k, v, off, stream=r)  # at the same time
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want + want, a + b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = bsa.prompt_attention(q, k, v, off)
    q.mul_(0.5)
    off.copy_(ptr([0, 900, 100]).cuda())
    g.replay()
    want = bsa.prompt_attention(q, k, v, off)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals(bsa):
    x = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    off = ptr([8]).cuda()
    f = bsa.prompt_attention
    for bad in (lambda: f(x.float(), x, x, off), lambda: f(x.cpu(), x, x, off), lambda: f(x[0], x, x, off), lambda: f(x, x[:4], x[:4], off),
                lambda: f(x, x, x[:, :2], off), lambda: f(x, x.half(), x.half(), off), lambda: f(x.transpose(1, 2), x, x, off),
                lambda: f(x, x, x, off.long()), lambda: f(x, x, x, off.cpu()), lambda: f(x, x, x, off[:1]), lambda: f(x, x, x, off, out=x[:4]),
                lambda: f(x, x, x, off, lse=torch.zeros(4, 8, device="cuda")), lambda: f(x, x, x, off, workspace=torch.zeros(999, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    y = torch.zeros(8, 4, 96, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: f(y, y, y, off), lambda: f(x, x[:, :3], x[:, :3], off), lambda: f(x[:1].expand(8, 4, 64), x, x, off),
                lambda: f(x, x[:, :1].expand(8, 4, 64), x, off), lambda: f(x, x, x, off, out=x[:1].expand(8, 4, 64)),
                lambda: f(x, x, x, off, scale=math.nan), lambda: f(x, x, x, off, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(bsa.BsaError):
            bad()
    o, lse = f(x[:0], x[:0], x[:0], ptr([0]).cuda())
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)

@pytest.mark.parametrize("d,Hq,Hkv", [(64, 6, 3), (128, 6, 3)])
@pytest.mark.parametrize("lens", [[1500, 130, 7], [100], [2100]])
def test_values_of_any_finite_size(bsa, d, Hq, Hkv, lens):
    """bfloat16 values scaled by a power of two scale the outputs, bit for bit: sums of weights are below 1 in all, so
    that no finite value leaves fp32's range, with scores that rise, fall or jump after the first 128 keys."""
    gen = torch.Generator().manual_seed(d + len(lens))
    T = sum(lens)
    u = torch.randint(0, 2, (d,), generator=gen).double() * 2 - 1
    j = torch.arange(T).double()
    f = torch.stack([j / T * 5, 5 - j / T * 5, (j // 200 % 2) * 4], 1)
    k = (f[:, :, None] * u).to(torch.bfloat16)
    q = ((torch.rand(T, Hq, 1, generator=gen).double() + 0.25) * u * 8 / d ** 0.5).to(torch.bfloat16)
    v = rows(gen, T, Hkv, d, torch.bfloat16).clamp(-3.9, 3.9)
    for causal in (True, False):
        o, lse = check(bsa, q, k, v, ptr(lens), causal)
        for e in (115, 125, -90):
            big = (v.double() * 2.0 ** e).to(torch.bfloat16)
            assert big.isfinite().all()
            got, gl = bsa.prompt_attention(q.cuda(), k.cuda(), big.cuda(), ptr(lens).cuda(), causal=causal)
            assert torch.equal(gl, lse) and torch.equal(got.double(), o.double() * 2.0 ** e), e


def test_the_largest_values(bsa):
    """Every value the type's largest: the mean is that value (equal weights, their sums exact)."""
    top = torch.finfo(torch.bfloat16).max
    k = torch.zeros(1000, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, top)
    o, _ = bsa.prompt_attention(k, k, v, ptr([1000]).cuda())
    assert (o == top).all()


@pytest.mark.parametrize("n,T", [(3, 900), (70, 900)])
def test_what_any_block_records_is_reported(bsa, n, T):
    """Status words are each block's own: whatever the workspace held is gone after a call, and what one block recorded
    is not lost to another's."""
    gen = torch.Generator().manual_seed(n)
    x = rows(gen, T, 8, 64, torch.bfloat16).cuda()
    off = ptr([T // n] * (n - 1) + [T - T // n * (n - 1)]).cuda()
    ws = torch.full((bsa.prompt_workspace_bytes(n, T, 8, 8),), 0xFA, dtype=torch.uint8, device="cuda")
    bsa.prompt_attention(x, x, x, off, workspace=ws)
    assert bsa.prompt_status(ws) == (0, 0)
    words = ws.view(torch.int32)
    words[16 + 2 * 5:16 + 2 * 5 + 2] = torch.tensor([-6, 5 << 8 | 0x52], dtype=torch.int32)  # as block 5's wait would
    assert bsa.prompt_status(ws) == (-6, 5 << 8 | 0x52)
    bsa.prompt_attention(x, x, x, off, workspace=ws)
    assert bsa.prompt_status(ws) == (0, 0)


def test_without_lse(bsa):
    """LSE = NULL through the C ABI: the same outputs."""
    from block_sparse_attention_plan_gb300 import _prompt as P
    gen = torch.Generator().manual_seed(8)
    for d, lens in ((64, [200, 3]), (128, [5000, 60])):
        T = sum(lens)
        q, k, v = (rows(gen, T, h, d, torch.bfloat16).cuda() for h in (4, 2, 2))
        off = ptr(lens).cuda()
        want, _ = bsa.prompt_attention(q, k, v, off)
        out = torch.zeros_like(q)
        ws = torch.empty(bsa.prompt_workspace_bytes(2, T, 4, 2), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        r = [ctypes.byref(P.RowsC(x.data_ptr(), 0, d, x.shape[1] * d)) for x in (q, k, v, out)]
        assert P._library().bsa_prompt_attention(*r, None, 0, off.data_ptr(), 2, T, 4, 2, d, 1, 0.0, ws.data_ptr(), ws.numel(), None) == 0
        assert bsa.prompt_status(ws) == (0, 0) and torch.equal(out, want)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 7, 1), (128, 8, 2)])
@pytest.mark.parametrize("lens", [[4096], [4000] + [1] * 60 + [0, 17, 19], [20] * 64, [0] * 30 + [4033] + [63] + [0] * 30])
def test_with_and_without_the_schedule(bsa, d, Hq, Hkv, lens):
    """Up to 64 prompts of 4096 tokens find their items without the schedule kernel: at the border, and one prompt or
    token past it, with a long prompt ahead of short ones and behind, the same bits."""
    gen = torch.Generator().manual_seed(len(lens))
    T = sum(lens)
    q, k, v = (rows(gen, 4097, h, d, torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
    for causal in (True, False):
        few = bsa.prompt_attention(q[:T], k[:T], v[:T], ptr(lens).cuda(), causal=causal)
        more = bsa.prompt_attention(q[:T], k[:T], v[:T], ptr(lens + [0] * (65 - len(lens))).cuda(), causal=causal)
        longer = bsa.prompt_attention(q, k, v, ptr(lens).cuda(), causal=causal)      # (rows of no prompt behind)
        for other in (more, longer):
            assert torch.equal(few[0], other[0][:T]) and torch.equal(few[1], other[1][:T])
    if T > 3000:
        return
    check(bsa, *(x[:T].cpu() for x in (q, k, v)), ptr(lens))


def test_rows_past_32_bit_offsets(bsa):
    """Rows whose offsets pass 2^31 elements and 2^32 bytes: by far tokens, by far heads, and outputs so."""
    gen = torch.Generator().manual_seed(9)
    T, H, d = 300, 4, 64
    far = (1 << 31) // 100 // 8 * 8                        # elements between tokens: T of them pass 2^32
    room = torch.zeros(T * far + H * d, dtype=torch.bfloat16, device="cuda")
    x = rows(gen, T, H, d, torch.bfloat16).cuda()
    for shape in ((far, d), (d, far * 64)):                # (by tokens, by heads)
        view = room.as_strided((T, H, d), (*shape, 1))
        view.copy_(x)
        off = ptr([170, 130]).cuda()
        want, wl = bsa.prompt_attention(x, x[:, :2], x[:, 2:], off)
        got, gl = bsa.prompt_attention(view, view[:, :2], view[:, 2:], off)
        assert torch.equal(want, got) and torch.equal(wl, gl)
        r = bsa.rope_create(64)
        tq, tk = bsa.rope(r, x, x[:, :2])
        gq, gk = bsa.rope(r, view, view[:, :2], out_q=torch.empty_like(x), out_k=torch.empty_like(x[:, :2]))
        assert torch.equal(tq, gq) and torch.equal(tk, gk)
        bsa.rope(r, view, out_q=view)
        assert torch.equal(view, tq)
        bsa.prompt_attention(x, x[:, :2], x[:, 2:], off, out=view)
        assert torch.equal(view, want)
        view.zero_()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,g", [(64, 1), (64, 7), (128, 4), (128, 2)])
@pytest.mark.parametrize("lens", [[300], [700, 45, 523]])
def test_outputs_do_not_depend_on_rows_of_others(bsa, dtype, d, g, lens):
    """The same bits whatever rows lie ahead of a prompt and behind it: none, other prompts', or anything."""
    gen = torch.Generator("cuda").manual_seed(d + g)
    T, pad = sum(lens), 300
    q, k, v = (torch.randn(T + 2 * pad, h, d, device="cuda", generator=gen).to(dtype) for h in (2 * g, 2, 2))
    off = ptr(lens, pad)
    for causal in (True, False):
        want = bsa.prompt_attention(q, k, v, off.cuda(), causal=causal)
        for fill in (0.0, 100.0, math.inf, math.nan):
            a, b, c = q.clone(), k.clone(), v.clone()
            for x in (a, b, c):
                x[:pad] = fill
                x[pad + T:] = fill * torch.randn(x[pad + T:].shape, device="cuda", generator=gen).to(dtype)
            got = bsa.prompt_attention(a, b, c, off.cuda(), causal=causal)
            for w, o in zip(want, got):
                assert torch.equal(w[pad:pad + T], o[pad:pad + T]), (causal, fill)
        for i, n in enumerate(lens):  # each prompt on its own
            lo = off[i].item()
            alone = bsa.prompt_attention(q[lo:lo + n], k[lo:lo + n], v[lo:lo + n], ptr([n]).cuda(), causal=causal)
            for w, o in zip(want, alone):
                assert torch.equal(w[lo:lo + n], o), (causal, i)
