"""GPU tests of rotary positions (bsa_rope_apply) against fp64."""
import math

import numpy as np
import pytest
import torch

from oracle import prompt as OP

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def rows(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen).to(dtype)


def bound(x, ref, amp, dtype, rot):
    """Half a step of the type at the result, 2^-24 of the smallest fp16 steps, and the fp32 terms: sines and
    cosines are off by at most 2^-22 (their argument by pi 2^-25, the functions by 2^-23), the factor, products
    and the sum round four times at 2^-24 of |x_a| + |x_b| each."""
    a = np.abs(x)
    pair = np.zeros_like(a)
    for p, q in ((0, 1), (1, 0)):  # either pairing is covered by the row's two largest elements
        pair[..., :rot] = np.sort(a[..., :rot], -1)[..., -2:].sum(-1)[..., None]
    return np.abs(ref) * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 0) + amp * pair * (2.0 ** -22 + 4 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", ["half", "neighbours"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [
    (1, 1, 1, 0, 64, 16), (1, 1, 32, 8, 128, 128), (3, 5, 7, 1, 128, 64), (2, 129, 4, 4, 64, 64), (64, 1, 32, 8, 128, 96),
    (1, 700, 3, 2, 64, 48), (2, 2500, 9, 3, 128, 112)])
def test_against_the_oracle(bsa, dtype, pairs, B, T, Hq, Hk, d, rot):
    gen = torch.Generator().manual_seed(B * T + d)
    q, k = rows(gen, B, T, Hq, d, dtype=dtype), rows(gen, B, T, max(Hk, 1), d, dtype=dtype)
    pos = torch.randint(-5000, 1 << 20, (B, T), generator=gen, dtype=torch.int32)
    pos[0, 0] = (1 << 31) - 1
    pos[-1, -1] = -(1 << 31) if B * T > 1 else 0
    r = bsa.rope_create(rot, base=10000.0, pairs=pairs, scaling="parts", factor=4.0, original=2048)
    f, amp = OP.frequencies(rot, 10000.0, "parts", 4.0, 2048)
    qd, kd = q.cuda().transpose(1, 2), k.cuda().transpose(1, 2)  # strided
    for inverse in (False, True):
        oq, ok = bsa.rope(r, qd, kd if Hk else None, positions=pos.cuda(), inverse=inverse)
        assert oq.shape == qd.shape and oq.dtype == dtype
        for x, o in ((qd, oq), (kd, ok)):
            if o is None:
                continue
            x = x.double().cpu().numpy()
            ref = OP.rotate(x, pos.numpy()[:, None], f, amp, pairs, inverse)
            off = np.abs(o.double().cpu().numpy() - ref)
            assert (off <= bound(x, ref, amp, dtype, rot)).all(), off.max()
            assert np.array_equal(o.double().cpu().numpy()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling,factor,original", [("none", 1.0, 0), ("linear", 2.5, 0), ("base", 8.0, 0), ("parts", 16.0, 4096)])
def test_packed_and_without_positions(bsa, scaling, factor, original):
    gen = torch.Generator().manual_seed(1)
    q = rows(gen, 333, 6, 64, dtype=torch.bfloat16)
    r = bsa.rope_create(64, base=500000.0, scaling=scaling, factor=factor, original=original)
    f, amp = OP.frequencies(64, 500000.0, scaling, factor, original)
    o, none = bsa.rope(r, q.cuda())
    assert none is None
    x = q.double().numpy().transpose(1, 0, 2)
    ref = OP.rotate(x, np.arange(333), f, amp)
    assert (np.abs(o.double().cpu().numpy().transpose(1, 0, 2) - ref) <= bound(x, ref, amp, torch.bfloat16, 64)).all()
    # the same by positions, and batched
    p, _ = bsa.rope(r, q.cuda().unsqueeze(0).transpose(1, 2), positions=torch.arange(333, dtype=torch.int32, device="cuda").view(1, -1))
    assert torch.equal(p[0].transpose(0, 1), o)


def test_in_place_and_into_slices(bsa):
    gen = torch.Generator().manual_seed(2)
    r = bsa.rope_create(32, pairs="neighbours")
    qkv = rows(gen, 100, 12, 128, dtype=torch.float16).cuda()  # heads 0-7 q, 8-9 k, 10-11 v of one projection
    q, k = qkv[:, :8], qkv[:, 8:10]
    want = [t.clone() for t in bsa.rope(r, q.contiguous(), k.contiguous())]
    before = qkv.clone()
    big = torch.full((102, 2, 128), 3.0, dtype=torch.float16, device="cuda")
    bsa.rope(r, q, k, out_q=q, out_k=big[1:101])
    assert torch.equal(qkv[:, :8], want[0]) and torch.equal(big[1:101], want[1])
    assert torch.equal(qkv[:, 8:], before[:, 8:]) and (big[0] == 3).all() and (big[101] == 3).all()
    bsa.rope(r, k, out_q=k)
    assert torch.equal(qkv[:, 8:10], want[1]) and torch.equal(qkv[:, 10:], before[:, 10:])


@pytest.mark.parametrize("pairs", ["half", "neighbours"])
def test_inverse_is_the_gradient(bsa, pairs):
    """Against the transpose in fp64, and against differences of the operator in its own arithmetic: a step along one
    element moves the outputs by the column of the matrix that the inverse reads as a row."""
    gen = torch.Generator().manual_seed(3)
    r = bsa.rope_create(48, pairs=pairs, scaling="parts", factor=8.0, original=100)
    f, amp = OP.frequencies(48, 10000.0, "parts", 8.0, 100)
    gy = rows(gen, 5, 2, 64, dtype=torch.float16)
    pos = torch.tensor([0, 3, 70, 5000, 99999], dtype=torch.int32)
    gx, _ = bsa.rope(r, gy.cuda(), positions=pos.cuda(), inverse=True)
    eye = torch.eye(64, dtype=torch.float16).view(64, 1, 64)  # every unit step at once
    for t in range(5):
        cols, _ = bsa.rope(r, eye.cuda(), positions=torch.full((64,), int(pos[t]), dtype=torch.int32, device="cuda"))
        A = cols[:, 0].double().cpu().numpy()                 # A[i] = y(e_i) - y(0)
        g = gy[t].double().numpy()
        want = g @ A.T
        # A's elements are rounded to fp16 (2^-11), two of them a sum; the result once more
        assert np.abs(gx[t].double().cpu().numpy() - want).max() <= 4 * 2.0 ** -11 * amp * np.abs(g).max() + 2.0 ** -11 * np.abs(want).max()
    x = gy.double().numpy().transpose(1, 0, 2)
    ref = OP.rotate(x, pos.numpy(), f, amp, pairs, inverse=True)
    assert (np.abs(gx.double().cpu().numpy().transpose(1, 0, 2) - ref) <= bound(x, ref, amp, torch.float16, 48)).all()


def test_other_stream_and_a_graph(bsa):
    gen = torch.Generator().manual_seed(4)
    r = bsa.rope_create(128)
    q, k = (rows(gen, 40, h, 128, dtype=torch.bfloat16).cuda() for h in (8, 2))
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    want = [t.clone() for t in bsa.rope(r, q, k, positions=pos)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bsa.rope(r, q, k, positions=pos, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = bsa.rope(r, q, k, positions=pos)
    q.add_(1.0)
    pos.add_(7)
    g.replay()
    want = bsa.rope(r, q, k, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(bsa):
    r = bsa.rope_create(64)
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: bsa.rope(r, q.float()), lambda: bsa.rope(r, q.cpu()), lambda: bsa.rope(r, q[0]), lambda: bsa.rope(r, q.transpose(1, 2)),
                lambda: bsa.rope(r, q, q[:3]), lambda: bsa.rope(r, q, q.half()), lambda: bsa.rope(r, q, q.unsqueeze(0)),
                lambda: bsa.rope(r, q, positions=pos[:3]), lambda: bsa.rope(r, q, positions=pos.long()),
                lambda: bsa.rope(r, q, positions=pos.cpu()), lambda: bsa.rope(r, q, out_q=q[:3]),
                lambda: bsa.rope(r, q.unsqueeze(0).transpose(1, 2), positions=pos), lambda: bsa.rope_create(64, pairs="both"),
                lambda: bsa.rope_create(64, scaling="all")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bsa.BsaError):
        bsa.rope_create(60)
    with pytest.raises(bsa.BsaError):
        bsa.rope(bsa.rope_create(128), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(bsa.BsaError):  # rows that would be written twice
        bsa.rope(r, q, out_q=q[:1].expand(4, 2, 128))
    assert bsa.rope(r, q[:0])[0].shape == (0, 2, 128)
    o, ok = bsa.rope(r, q, q[:, :0])  # no key heads
    assert ok.shape == (4, 0, 128) and torch.equal(o, q)


def test_an_output_for_keys_that_are_not_given_is_refused(bsa):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        bsa.rope(bsa.rope_create(64), q, out_k=q.clone())


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("inverse", [True, False])
def test_gradients_reach_the_inputs(bsa, packed, inverse):
    """The result belongs to the graph of its inputs: their gradients are the outputs' turned the other way."""
    gen = torch.Generator().manual_seed(7)
    shape = lambda h: (60, h, 64) if packed else (3, h, 20, 64)
    q, k = (rows(gen, *shape(h), dtype=torch.bfloat16).cuda().requires_grad_() for h in (4, 2))
    gq, gk = (rows(gen, *shape(h), dtype=torch.bfloat16).cuda() for h in (4, 2))
    pos = torch.randint(0, 9999, (60,) if packed else (3, 20), generator=gen).int().cuda()
    r = bsa.rope_create(32, pairs="neighbours", scaling="parts", factor=4.0, original=100)
    oq, ok = bsa.rope(r, q, k, positions=pos, inverse=inverse)
    with torch.no_grad():
        wq, wk = bsa.rope(r, q, k, positions=pos, inverse=inverse)
        tq, tk = bsa.rope(r, gq, gk, positions=pos, inverse=not inverse)
    assert not wq.requires_grad and torch.equal(oq, wq) and torch.equal(ok, wk)
    got = torch.autograd.grad((oq, ok), (q, k), (gq, gk))
    assert torch.equal(got[0], tq) and torch.equal(got[1], tk)
    # one of two; an expanded gradient; rows of another order; no keys
    a, _ = bsa.rope(r, q, k.detach(), positions=pos, inverse=inverse)
    assert torch.equal(torch.autograd.grad(a.sum(), q)[0], bsa.rope(r, torch.ones_like(gq), positions=pos, inverse=not inverse)[0])
    _, b = bsa.rope(r, q.detach(), k, positions=pos, inverse=inverse)
    assert torch.equal(torch.autograd.grad(b, k, gk.transpose(0, 1).contiguous().transpose(0, 1))[0], tk)
    c, none = bsa.rope(r, q, positions=pos, inverse=inverse)
    assert none is None and torch.equal(torch.autograd.grad(c, q, gq)[0], tq)
    # and through a projection whose heads q and k are
    x = rows(gen, *shape(6), dtype=torch.bfloat16).cuda().requires_grad_()
    axis = 1
    y = x * 1
    oq, ok = bsa.rope(r, y.narrow(axis, 0, 4), y.narrow(axis, 4, 2), positions=pos, inverse=inverse)
    torch.autograd.backward((oq, ok), (gq, gk))
    assert torch.equal(x.grad, torch.cat([tq, tk], axis))


def test_outputs_given_to_a_call_with_gradients_are_refused(bsa):
    r = bsa.rope_create(64)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = q * 1
    for bad in (lambda: bsa.rope(r, y, out_q=y), lambda: bsa.rope(r, y.detach(), y, out_k=torch.empty_like(y)),
                lambda: bsa.rope(r, y, out_q=torch.empty_like(y))):
        with pytest.raises(ValueError):
            bad()
    with torch.no_grad():
        assert bsa.rope(r, y, out_q=y)[0] is y


def test_gradients_in_a_captured_graph(bsa):
    """Forward and gradients captured together.  (No eager graph of the same leaves may be alive then, whatever its
    operations: a leaf's node belongs to the stream on which it was made, and capture refuses to wait for it.)"""
    gen = torch.Generator().manual_seed(8)
    r = bsa.rope_create(64)
    q, gy = (rows(gen, 30, 4, 64, dtype=torch.bfloat16).cuda() for _ in range(2))
    q.requires_grad_()
    pos = torch.arange(30, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # (the first gradient sets up the engine)
        torch.autograd.grad(bsa.rope(r, q, positions=pos)[0], q, gy)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, _ = bsa.rope(r, q, positions=pos)
        gx, = torch.autograd.grad(o, q, gy)
    with torch.no_grad():
        q.mul_(2.0)
        gy.add_(1.0)
        pos.add_(5)
        g.replay()
        assert torch.equal(o, bsa.rope(r, q, positions=pos)[0]) and torch.equal(gx, bsa.rope(r, gy, positions=pos, inverse=True)[0])
