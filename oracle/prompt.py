"""fp64 oracle of the operators on prompts' rows: rotary positions and the
attention of packed prompts.  Shares no code with the CUDA path.  Test
infrastructure only."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0):
    """Radians per position of each pair, and the amplitude."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    out, amp = [], 1.0
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            turns = original * f / (2 * math.pi)
            stay = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            f = (1 - stay) * f / factor + stay * f
            amp = 0.1 * math.log(factor) + 1.0
        out.append(f)
    return np.array(out), amp


def rotate(x, positions, freqs, amp=1.0, pairs="half", inverse=False):
    """x [..., T, d] fp64 at positions [..., T] (broadcast against x's leading axes)."""
    y = np.array(x, dtype=np.float64)
    r = 2 * len(freqs)
    a = np.asarray(positions, dtype=np.float64)[..., None] * freqs
    co, si = amp * np.cos(a), amp * np.sin(a) * (-1 if inverse else 1)
    for i in range(r // 2):
        p, q = (i, i + r // 2) if pairs == "half" else (2 * i, 2 * i + 1)
        u, v = np.array(x[..., p], dtype=np.float64), np.array(x[..., q], dtype=np.float64)
        y[..., p] = u * co[..., i] - v * si[..., i]
        y[..., q] = v * co[..., i] + u * si[..., i]
    return y


def attention(q, k, v, offsets, causal=True, scale=None):
    """q [T, Hq, d], k, v [T, Hkv, d] fp64: O [T, Hq, d], LSE [T, Hq], and for error bounds
    sum_j w_j |v_j| and the largest sum_d |q_d k_d| * scale of each row.  Rows of no prompt
    are NaN."""
    T, Hq, d = q.shape
    g = Hq // k.shape[1]
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    O, A = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, mag = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for a, b in zip(offsets[:-1], offsets[1:]):
        for h in range(Hq):
            for i in range(a, b):
                e = i + 1 if causal else b
                s = k[a:e, h // g] @ q[i, h] * sc
                m = s.max()
                w = np.exp(s - m)
                t = w.sum()
                O[i, h] = (w / t) @ v[a:e, h // g]
                A[i, h] = (w / t) @ np.abs(v[a:e, h // g])
                lse[i, h] = m + math.log(t)
                mag[i, h] = (np.abs(k[a:e, h // g]) @ np.abs(q[i, h])).max() * sc
    return O, lse, A, mag
