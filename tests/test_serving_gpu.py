"""GPU test of the operators from a prompt to a cache of bounded size together, as a
server runs them: rotary positions, attention of packed prompts, storing, weights of the
prompts' last queries, eviction, then steps of decoding with weights and evictions."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as OC
from oracle import prompt as OP
from test_evict_gpu import assert_state, i32
from test_prompt_gpu import bounds, ptr

pytestmark = pytest.mark.gpu


def close_weights(got, want, m, H):
    for s in range(len(m.lens)):
        n = int(m.lens[s])
        g, w = got[s, :, :n].double().cpu().numpy(), want[s, :, :n]
        # each row's LSE is the attention kernel's (2^-20 of a few units), scores and sums as there; weights of
        # several calls add up
        assert np.allclose(g, w, rtol=2.0 ** -9, atol=2.0 ** -14), (s, np.abs(g - w).max())


@pytest.mark.parametrize("kind,d,dtype", [("e4m3", 64, torch.bfloat16), ("int8", 128, torch.float16)])
def test_prompts_to_a_bounded_cache(bsa, kind, d, dtype):
    gen = torch.Generator().manual_seed(d)
    Hq, H, page, sb = 8, 2, 32, 16
    lens = [150, 77, 200, 1]
    n, T = len(lens), sum(lens)
    budget = [64, 64, 96, 64]
    off = ptr(lens)
    q, k, v = ((torch.randn(T, h, d, generator=gen)).to(dtype).cuda() for h in (Hq, H, H))
    pos = torch.cat([torch.arange(x) for x in lens]).int().cuda()
    r = bsa.rope_create(d // 2, base=10000.0, scaling="parts", factor=4.0, original=64)
    f, amp = OP.frequencies(d // 2, 10000.0, "parts", 4.0, 64)
    rq, rk = bsa.rope(r, q, k, positions=pos)
    for x, y in ((q, rq), (k, rk)):
        ref = OP.rotate(x.double().cpu().numpy().transpose(1, 0, 2), pos.cpu().numpy(), f, amp).transpose(1, 0, 2)
        assert np.abs(y.double().cpu().numpy() - ref).max() <= np.abs(ref).max() * torch.finfo(dtype).eps / 2 + 2.0 ** -18
    o, lse = bsa.prompt_attention(rq, rk, v, off.cuda())
    O, L, A, mag = OP.attention(*(x.double().cpu().numpy() for x in (rq, rk, v)), off.numpy())
    to, tl = bounds(O, L, A, mag, dtype, max(lens), float(v.abs().max()))
    assert (np.abs(o.double().cpu().numpy() - O) <= to).all() and (np.abs(lse.double().cpu().numpy() - L) <= tl).all()

    # into the cache
    m = OC.CacheModel(40, H, page, d, n, 8, kind, sb, seed=1)
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    up = lambda a: torch.from_numpy(a.copy()).cuda()
    c = bsa.Cache(*(up(x).view(dt) for x in m.codes), *(up(x) for x in m.scales), up(m.table), up(m.lens), up(m.refs))
    bsa.cache_resize(c, i32(*lens))
    m.resize(lens)
    pad = lambda x: torch.stack([torch.nn.functional.pad(x[a:b].transpose(0, 1), (0, 0, 0, max(lens) - (b - a)))
                                 for a, b in zip(off.tolist(), off.tolist()[1:])])
    pk, pv = pad(rk), pad(v)
    bsa.cache_append(c, pk, pv, counts=i32(*lens))
    m.append(pk.double().cpu().numpy(), pv.double().cpu().numpy(), counts=lens)
    assert_state(c, m)

    # the last queries of each prompt look back
    nq = 16
    last = torch.stack([rq[[max(a, b - nq + i) for i in range(nq)]].transpose(0, 1) for a, b in zip(off.tolist(), off.tolist()[1:])])
    weights = torch.full((n, H, 256), math.nan, device="cuda")  # fresh tokens begin at 0 whatever lies there
    want = np.full((n, H, 256), np.nan)

    def look(queries, fresh):
        w = queries.shape[2]
        _, z = bsa.cache_attention(c, queries, causal=True)
        bsa.cache_weigh(c, queries, z, weights, causal=True, fresh=fresh)
        qd, zd = queries.double().cpu().numpy(), np.empty((n, Hq, w))
        for b in range(n):
            kk, vv = m.values(b)
            see = np.array([[[j <= len(kk[0]) - w + i for j in range(len(kk[0]))] for i in range(w)]] * Hq)
            zd[b] = OC.attention(qd[b], kk, vv, see)[1]
        m.weigh(want, qd, zd, keep=lambda b, h, i, j: j <= m.lens[b] - w + i, fresh=max(w, fresh))
        close_weights(weights, want, m, H)

    def evict():
        ref = weights.cpu().numpy().copy()
        rows = m.evict(ref, budget, sink=4, recent=16)
        kept = bsa.cache_evict(c, weights, i32(*budget), sink=4, recent=16)
        assert_state(c, m)
        assert np.array_equal(weights.cpu().numpy(), ref, equal_nan=True)
        for b, rr in enumerate(rows):
            for h in range(H):
                assert kept[b, h, :len(rr[h])].tolist() == rr[h]
                want[b, h, :len(rr[h])] = want[b, h][rr[h]]

    look(last, 1 << 30)
    evict()
    assert bsa.cache_status(c) == (0, 0) and m.lens.tolist() == [64, 64, 96, 1]

    # decoding: a token of each sequence at its own position, eviction every third step
    at = torch.tensor(lens, dtype=torch.int32, device="cuda").view(-1, 1)
    for step in range(7):
        x = (torch.randn(n, h, 1, d, generator=gen).to(dtype).cuda() for h in (Hq, H, H))
        tq, tk, tv = x
        tq, tk = bsa.rope(r, tq, tk, positions=at)
        at += 1
        grown = [int(y) + 1 for y in m.lens]
        bsa.cache_resize(c, i32(*grown))
        m.resize(grown)
        bsa.cache_append(c, tk, tv)
        m.append(tk.double().cpu().numpy(), tv.double().cpu().numpy())
        assert_state(c, m)
        look(tq, 1)
        if step % 3 == 2:
            evict()
    assert bsa.cache_status(c) == (0, 0) and m.lens.tolist() == [65, 65, 97, 8]
