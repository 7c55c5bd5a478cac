"""fp64 / plain-Python oracle of the 8-bit paged K/V cache: a model of its
state (table, lengths, counts, codes, scales) with every operation written as
loops over sequences and tokens, and attention as the weighted mean it is.
Shares no code with the CUDA path.  Test infrastructure only."""
from __future__ import annotations

import math

import numpy as np

TOP = {"e4m3": 448.0, "int8": 127.0}
MIN_SCALE = 2.0 ** -100


def e4m3_values():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; 0x7f and 0xff are NaN, there are no infinities."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            x = math.nan
        out[c] = -x if s else x
    return out


_E4M3 = e4m3_values()


def decode(codes, kind):
    """fp64 values of uint8 / int8 codes."""
    if kind == "int8":
        return codes.astype(np.int8).astype(np.float64)
    return _E4M3[codes.view(np.uint8)]


def encode(x, kind):
    """Codes (uint8) nearest to x, ties to even, saturated; NaN is stored as
    NaN (e4m3) or 0 (int8)."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    x = np.clip(np.where(nan, 0.0, x), -TOP[kind], TOP[kind])
    if kind == "int8":
        return np.round(x).astype(np.int8).view(np.uint8)
    mag = _E4M3[:127]                       # 0 .. 448, ascending with the code
    hi = np.searchsorted(mag, np.abs(x))    # first value >= |x|
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.abs(x) - mag[lo], mag[hi] - np.abs(x)
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def scale_for(amax, kind):
    """Smallest power of two, at least 2^-100, that takes amax into range."""
    s = MIN_SCALE
    while amax > TOP[kind] * s:
        s *= 2.0
    return s


class CacheModel:
    def __init__(self, num_pages, heads, page, d, max_seqs, max_pages, kind="e4m3", sb=None, seed=0):
        rng = np.random.default_rng(seed)
        self.kind, self.page, self.sb, self.d = kind, page, sb or min(page, 64), d
        shape = (num_pages, heads, page, d)
        # Anything may lie in pages no token has been stored in.
        self.codes = [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
        self.scales = [rng.standard_normal((num_pages, heads, page // self.sb)).astype(np.float32) for _ in range(2)]
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.lens = np.zeros(max_seqs, np.int32)
        self.refs = np.zeros(num_pages, np.int32)

    # ---- pages
    def _pages(self, n):
        return -(-n // self.page)

    def resize(self, new_lens, seqs=None):
        """Returns the number of pages missing (then nothing has changed)."""
        seqs = range(len(new_lens)) if seqs is None else seqs
        refs, table = self.refs.copy(), self.table.copy()
        items = [(int(s), int(n)) for s, n in zip(seqs, new_lens) if s >= 0]
        for s, n in items:
            for j in range(self._pages(n), self._pages(self.lens[s])):
                refs[table[s, j]] -= 1
                table[s, j] = -1
        free = [p for p in range(len(refs)) if refs[p] == 0]
        copies, need = [], 0
        for s, n in items:
            have = int(self.lens[s])
            take = []
            if n > have and have % self.page:
                j = have // self.page
                if refs[table[s, j]] > 1:
                    take.append((j, table[s, j]))
            take += [(j, None) for j in range(self._pages(have), self._pages(n))]
            for j, old in take:
                need += 1
                if need > len(free):
                    continue
                p = free[need - 1]
                if old is not None:
                    refs[old] -= 1
                    copies.append((old, p))
                refs[p] = 1
                table[s, j] = p
        if need > len(free):
            return need - len(free)
        for old, p in copies:
            for x in self.codes + self.scales:
                x[p] = x[old]
        self.refs, self.table = refs, table
        for s, n in items:
            have = int(self.lens[s])
            if n > have + 1:  # blocks wholly past the old length hold nothing yet: scale 0
                for b in range(-(-have // self.sb), self._pages(n) * self.page // self.sb):
                    for x in self.scales:
                        x[table[s, b * self.sb // self.page], :, b % (self.page // self.sb)] = 0
            self.lens[s] = n
        return 0

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            if a < 0 or b < 0:
                continue
            for j in range(self._pages(self.lens[a])):
                self.table[b, j] = self.table[a, j]
                self.refs[self.table[a, j]] += 1
            self.lens[b] = self.lens[a]

    def compact(self):
        L = int((self.refs > 0).sum())
        holes = [p for p in range(L) if self.refs[p] == 0]
        moved = [p for p in range(L, len(self.refs)) if self.refs[p] > 0]
        for p, to in zip(moved, holes):
            for x in self.codes + self.scales:
                x[to] = x[p]
            self.refs[to], self.refs[p] = self.refs[p], 0
            self.table[self.table == p] = to
        return L

    # ---- tokens
    def append(self, k, v, seqs=None, counts=None, start=None):
        """k, v [n, heads, T, d] (any float type's values)."""
        n, heads, T, _ = k.shape
        for i in range(n):
            s = i if seqs is None else int(seqs[i])
            c = T if counts is None else int(counts[i])
            if s < 0 or c == 0:
                continue
            at = int(self.lens[s]) - c if start is None else int(start[i])
            a = at
            while a < at + c:
                b = min(at + c, (a // self.sb + 1) * self.sb)
                b0 = a // self.sb * self.sb
                page, r0 = int(self.table[s, a // self.page]), b0 % self.page
                if self.refs[page] > 1:  # other sequences' too: left as it is
                    a = b
                    continue
                others = [t - b0 for t in range(b0, min(b0 + self.sb, int(self.lens[s]))) if not a <= t < b]
                for w, x in enumerate((k, v)):
                    for h in range(heads):
                        new = np.asarray(x[i, h, a - at:b - at], dtype=np.float64)
                        fin = np.abs(new[np.isfinite(new)])
                        sc = scale_for(fin.max() if fin.size else 0.0, self.kind)
                        rows = self.codes[w][page, h, r0:r0 + self.sb]
                        if others:
                            was = float(self.scales[w][page, h, r0 // self.sb])
                            if 0 < was < math.inf:
                                sc = max(sc, was)
                                if sc != was:
                                    rows[others] = encode(decode(rows[others], self.kind) * (was / sc), self.kind)
                            else:  # nothing is stored in the block yet
                                rows[others] = 0
                        rows[a - b0:b - b0] = encode(new / sc, self.kind)
                        self.scales[w][page, h, r0 // self.sb] = sc
                a = b

    # ---- weights and eviction
    def weigh(self, weights, q, lse, seqs=None, keep=None, fresh=0, scale=None):
        """weights[s, h, j] (fp64 array, in place) gather exp(scale q.K_j - lse) over the
        group's rows; q [B, Hq, nq, d], lse [B, Hq, nq], keep(b, h, i, j) -> bool."""
        B, Hq, nq, d = q.shape
        g = Hq // weights.shape[1]
        sc = 1.0 / math.sqrt(d) if scale is None else scale
        for b in range(B):
            s = b if seqs is None else int(seqs[b])
            if s < 0:
                continue
            n = int(self.lens[s])
            k = self.values(s)[0]
            weights[s, :, max(0, n - fresh):n] = 0
            for h in range(Hq):
                for i in range(nq):
                    z = float(lse[b, h, i])
                    if z == -math.inf:
                        continue
                    p = np.exp(sc * (k[h // g] @ q[b, h, i]) - z)
                    see = np.ones(n, bool) if keep is None else np.array([keep(b, h, i, j) for j in range(n)], bool)
                    weights[s, h // g, :n] += np.where(see, p, 0.0)

    def evict(self, weights, budgets, seqs=None, sink=0, recent=0):
        """Cuts sequences to budgets; `weights` [max_seqs, heads, tokens] in place.
        Returns the kept positions, [rows][heads] lists."""
        out = []
        for i, k in enumerate(budgets):
            s, k = i if seqs is None else int(seqs[i]), int(k)
            heads = weights.shape[1]
            if s < 0:
                out.append(None)
                continue
            n = int(self.lens[s])
            if n <= k:
                out.append([list(range(n))] * heads)
                continue
            r = min(recent, k)
            a = min(sink, k - r)
            rows = []
            for h in range(heads):
                w = weights[s, h]
                between = sorted(range(a, n - r), key=lambda j: (math.isnan(w[j]), -w[j] if w[j] == w[j] else 0.0, j))
                stay = list(range(a)) + sorted(between[:k - r - a]) + list(range(n - r, n))
                rows.append(stay)
                weights[s, h, :k] = w[stay].copy()
                at = lambda j: (int(self.table[s, j // self.page]), h, j % self.page)
                for codes, scales in zip(self.codes, self.scales):
                    of = lambda j: float(scales[at(j)[0], h, at(j)[2] // self.sb])
                    got = [(codes[at(j)].copy(), of(j)) for j in stay]
                    for b0 in range(0, k, self.sb):
                        b1 = min(k, b0 + self.sb)
                        if stay[b0:b1] == list(range(b0, b1)):
                            continue
                        good = [sc for _, sc in got[b0:b1] if 0 < sc < math.inf]
                        top = max(good, default=0.0)
                        for j in range(b0, b1):
                            c, sc = got[j]
                            if not 0 < sc < math.inf:
                                c = np.zeros_like(c)
                            elif sc != top:
                                c = encode(decode(c, self.kind) * (sc / top), self.kind)
                            codes[at(j)] = c
                        scales[at(b0)[0], h, at(b0)[2] // self.sb] = top
            for j in range(self._pages(k), self._pages(n)):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = k
            out.append(rows)
        return out

    def values(self, seq):
        """fp64 (K, V), each [heads, length, d], of a sequence."""
        n = int(self.lens[seq])
        out = []
        for codes, scales in zip(self.codes, self.scales):
            x = np.zeros((codes.shape[1], n, self.d))
            for j in range(self._pages(n)):
                p, a = int(self.table[seq, j]), j * self.page
                w = decode(codes[p], self.kind) * scales[p].astype(np.float64).repeat(self.sb, 1)[..., None]
                x[:, a:a + self.page] = w[:, :n - a]
            out.append(x)
        return out


def attention(q, k, v, keep, scale=None):
    """q [Hq, nq, d], k, v [Hkv, n, d] fp64, keep bool [Hq, nq, n].  Returns O,
    LSE, sum_j w_j |v_j| and the largest sum_d |q_d k_d| * scale over the kept
    keys of each row (for error bounds); empty rows give 0 and -inf."""
    Hq, nq, d = q.shape
    g = Hq // k.shape[0]
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    O, A = np.zeros((Hq, nq, d)), np.zeros((Hq, nq, d))
    lse, mag = np.full((Hq, nq), -np.inf), np.zeros((Hq, nq))
    for h in range(Hq):
        kk, vv = k[h // g], v[h // g]
        for i in range(nq):
            J = np.nonzero(keep[h, i])[0]
            if J.size == 0:
                continue
            s = kk[J] @ q[h, i] * sc
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            O[h, i], A[h, i] = w @ vv[J], w @ np.abs(vv[J])
            lse[h, i] = m + math.log(e.sum())
            mag[h, i] = (np.abs(kk[J]) @ np.abs(q[h, i])).max() * sc
    return O, lse, A, mag
