"""Cases of the operators from a prompt to a cache of bounded size: rotary positions of queries and keys, causal
attention of packed prompts, the attention weight that each cached token gathers, and the eviction of the tokens
that gathered least.

Packed rows: prompt i of a batch has rows offsets[i] .. offsets[i + 1] of q [T, Hq, d], k and v [T, Hkv, d]. The
cache is two pools of codes [pages, Hkv, page, d] (e4m3 or int8), an fp32 scale for each block of `sb` tokens of a
page and head, a page table [sequences, pages per sequence] (-1: none), a length per sequence and a reference count
per page; a value is code * scale. Gathered weights are fp32 [sequences, Hkv, tokens].
"""
import math

import torch

own = False

E4M3, INT8 = "e4m3", "int8"
CODE = {E4M3: torch.float8_e4m3fn, INT8: torch.int8}
TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a serving batch, far into long contexts: a token of each sequence.
        dict(name="rope_step", op="rope", n=64, T=1, Hq=32, Hkv=8, d=128, rot=128, pairs="half", base=500000.0, scaling="none",
             factor=1.0, original=0, far=120000, inverse=False, dtype="bf16"),
        # Packed prompts of one batch, positions scaled for a context longer than the trained one.
        dict(name="rope_prompt", op="rope", n=0, T=16001, Hq=32, Hkv=8, d=128, rot=128, pairs="half", base=10000.0,
             scaling="parts", factor=8.0, original=8192, far=60000, inverse=False, dtype="bf16"),
        # The gradients of a training step through neighbouring pairs in half of the head.
        dict(name="rope_back", op="rope", n=3, T=2047, Hq=16, Hkv=16, d=64, rot=32, pairs="neighbours", base=10000.0,
             scaling="linear", factor=4.0, original=0, far=2048, inverse=True, dtype="fp16"),
        # Short questions to a chat service, one of them empty: the latency of a call.
        dict(name="prompt_short", op="prompt", n=24, lo=0, hi=60, Hq=32, Hkv=8, d=128, causal=True, dtype="bf16"),
        # A batch of documents of unequal lengths, seven heads to a key head.
        dict(name="prompt_batch", op="prompt", n=6, lo=300, hi=4500, Hq=28, Hkv=4, d=64, causal=True, dtype="fp16"),
        # One long prompt.
        dict(name="prompt_long", op="prompt", n=1, lo=12007, hi=12007, Hq=32, Hkv=8, d=128, causal=True, dtype="bf16"),
        # One user, a short context: the latency of a call.
        dict(name="weigh_one", op="weigh", kind=E4M3, n=1, nq=1, Hq=32, Hkv=8, d=128, page=64, sb=64, lo=900, hi=901, causal=False,
             bk=0, topk=0, fresh=1),
        # A decode step of a serving batch of mixed context lengths.
        dict(name="weigh_batch", op="weigh", kind=E4M3, n=32, nq=1, Hq=32, Hkv=8, d=128, page=64, sb=64, lo=500, hi=32768,
             causal=False, bk=0, topk=0, fresh=1),
        # The last queries of several prompts look back over them, before their first eviction.
        dict(name="weigh_window", op="weigh", kind=INT8, n=4, nq=32, Hq=32, Hkv=8, d=64, page=16, sb=16, lo=3000, hi=12001,
             causal=True, bk=0, topk=0, fresh=1 << 30),
        # A batch of decoding sequences back to its budget.
        dict(name="evict_step", op="evict", kind=E4M3, n=32, Hkv=8, d=128, page=64, sb=64, lo=2177, hi=2304, keep=2048, sink=4,
             recent=256),
        # Many prompts of unequal lengths cut to one budget, some of them below it.
        dict(name="evict_many", op="evict", kind=INT8, n=48, Hkv=8, d=64, page=16, sb=16, lo=700, hi=12000, keep=1000, sink=1,
             recent=64),
        # One very long prompt, an eighth of it kept.
        dict(name="evict_prompt", op="evict", kind=E4M3, n=1, Hkv=8, d=128, page=64, sb=64, lo=64001, hi=64001, keep=8000, sink=16,
             recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "prompt", "prompt", "weigh", "weigh", "evict", "evict"])
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 7, 8])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        n = rng.choice([0, _log(rng, 1, 64)])
        T = _log(rng, 1, 16000 // max(n, 1))
        scaling = rng.choice(["none", "linear", "base", "parts"])
        return dict(op=op, n=n, T=T, Hq=Hkv * g if Hkv * g <= 32 else Hkv, Hkv=Hkv, d=d, rot=16 * rng.randint(1, d // 16),
                    pairs=rng.choice(["half", "neighbours"]), base=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.uniform(1.5, 16.0), original=rng.choice([4096, 8192]),
                    far=_log(rng, 1, 1000000), inverse=rng.random() < 0.3, dtype=dtype)
    if op == "prompt":
        n, Hq = _log(rng, 1, 32), Hkv * g if Hkv * g <= 32 else Hkv
        hi = _log(rng, 1, int(math.sqrt(4.0e9 / (n * Hq))))
        hi = min(hi, 12000)
        return dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, Hq=Hq, Hkv=Hkv, d=d, causal=rng.random() < 0.8, dtype=dtype)
    page = rng.choice([16, 32, 64, 128])
    c = dict(op=op, kind=rng.choice([E4M3, INT8]), n=_log(rng, 1, 64), Hkv=Hkv, d=d, page=page,
             sb=rng.choice([s for s in (16, 32, 64, 128) if s <= page]))
    if op == "weigh":
        hi = _log(rng, 70, max(100, min(60000, 1000000 // c["n"])))
        nq = rng.choice([1, 1, 1, 3, 8, 20])
        bk = rng.choice([0, 0, 32, 64, 128])
        return dict(c, nq=nq, Hq=Hkv * g if Hkv * g <= 32 else Hkv, lo=rng.randint(1, hi), hi=hi, causal=nq > 1, bk=bk,
                    topk=_log(rng, 1, 50) if bk else 0, fresh=rng.choice([0, nq, 1 << 30]))
    hi = _log(rng, 70, max(100, min(60000, 500000 // c["n"])))
    keep = _log(rng, 1, hi)
    return dict(c, lo=rng.randint(1, hi), hi=hi, keep=keep, sink=rng.randint(0, 20), recent=rng.randint(0, keep))


def _lens(c):
    """Lengths spread over [lo, hi]: the same for every seed."""
    return [c["lo"] + int((c["hi"] - c["lo"]) * ((i * 0.618034 + 0.9) % 1.0)) for i in range(c["n"])]


def _picked(c, n):
    """Key blocks that a group of heads reads of a sequence's n: a sink, a window of 16 and `topk` of the rest for each head."""
    rest = max(0, n - 17)
    k = min(c["topk"], rest)
    return min(n, 17), rest * (1 - (1 - k / rest) ** (c["Hq"] // c["Hkv"])) if rest else 0.0, k


def work(c):
    d, H = c["d"], c["Hkv"]
    if c["op"] == "rope":
        rows = max(c["n"], 1) * c["T"]
        return {"bytes": rows * (4 + 2 * 2 * d * (c["Hq"] + H)), "flops": 3 * rows * c["rot"] * (c["Hq"] + H)}
    if c["op"] == "prompt":
        lens = _lens(c)
        pairs = sum(n * (n + 1) / 2 if c["causal"] else n * n for n in lens)
        return {"bytes": sum(lens) * (4 * d * (c["Hq"] + H) + 4 * c["Hq"]) + 4 * c["n"], "flops": 4 * d * c["Hq"] * pairs}
    if c["op"] == "weigh":
        rows, keys, pairs, sums = c["Hq"] * c["nq"], 0.0, 0.0, 0.0
        for n in _lens(c):
            old = max(0, n - c["fresh"])  # tokens whose weight is read
            if c["bk"]:
                fixed, union, k = _picked(c, -(-n // c["bk"]))
                read = min(n, (fixed + union) * c["bk"])
                keys += read
                pairs += rows * min(n, (fixed + k) * c["bk"])
                sums += min(old, read) + max(read, n - old)
            else:
                keys += n
                pairs += rows * n
                sums += n + old
        return {"bytes": H * (keys * (d + 4 / c["sb"]) + 4 * sums) + c["n"] * rows * (2 * d + 4), "flops": 2 * d * pairs}
    cut = [n for n in _lens(c) if n > c["keep"]]
    moved = len(cut) * max(0, c["keep"] - c["sink"])
    scales = len(cut) * c["keep"] * 8 / c["sb"]
    return {"bytes": H * (4 * sum(cut) + 2 * moved * (2 * d + 4) + 2 * scales + 4 * len(cut) * c["keep"]) + 4 * c["n"], "flops": 0}


# ------------------------------------------------------------------------------------ inputs

def _frequencies(c):
    """Radians per position of each pair of a rotated row, as the scaling leaves them, and the factor on its values."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    base, s = c["base"], c["factor"]
    if c["scaling"] == "base":
        base = base * s ** (c["rot"] / max(c["rot"] - 2, 1))
    f = base ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "parts":  # pairs that turn often over the trained context stay, those that hardly turn are stretched
        stay = ((c["original"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        return f / s * (1 - stay) + f * stay, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _codes(gen, pages, c):
    """Codes and scales of pages whose blocks differ in magnitude. One page more than asked for: the plain form writes
    there what goes nowhere."""
    H, S, d, sb = c["Hkv"], c["page"], c["d"], c["sb"]
    codes = torch.empty(pages + 1, H, S, d, dtype=CODE[c["kind"]], device="cuda")
    step = max(1, (1 << 26) // (H * S * d))
    for a in range(0, pages + 1, step):
        x = torch.randn(min(step, pages + 1 - a), H, S, d, device="cuda", generator=gen)
        codes[a:a + step] = (x * 100).clamp(-448, 448).to(CODE[E4M3]) if c["kind"] == E4M3 else (x * 28).round().clamp(-127, 127).to(torch.int8)
    e = torch.randint(0, 2, (pages + 1, H, S // sb), device="cuda", generator=gen)
    return codes, torch.exp2(e - (7.0 if c["kind"] == E4M3 else 5.0))


def _cache(gen, c, lens):
    """A cache of sequences in shuffled pages: its tensors, and the framework's handle of them."""
    S = c["page"]
    held = [-(-n // S) for n in lens]
    pages = sum(held) + 2
    perm = torch.randperm(pages, device="cuda", generator=gen).int()
    table = torch.full((c["n"], max(held)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = perm[at:at + h]
        at += h
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[perm[:at].long()] = 1
    k, ks = _codes(gen, pages, c)
    v, vs = _codes(gen, pages, c)
    s = dict(c=c, k=k, v=v, ks=ks, vs=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), refs=refs)
    if own:
        import block_sparse_attention_plan_gb300 as bsa
        s["cache"] = bsa.Cache(k[:-1], v[:-1], ks[:-1], vs[:-1], table, s["lens"], refs)
    return s


def _blocks(gen, c, lens):
    """Per sequence and head: key block 0, the last 16 and `topk` of the others."""
    n = torch.tensor([-(-x // c["bk"]) for x in lens], device="cuda").view(-1, 1, 1)
    j = torch.arange(-(-max(lens) // c["bk"]), device="cuda")
    score = torch.rand(c["n"], c["Hq"], len(j), device="cuda", generator=gen)
    score = torch.where((j >= 1) & (j < n - 16), score, -1.0)
    best = torch.sort(score, -1, descending=True).values[..., min(c["topk"], len(j)) - 1].unsqueeze(-1)
    return ((j == 0) | ((j >= n - 16) & (j < n)) | ((score >= best) & (score >= 0))).to(torch.uint8)


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    if c["op"] == "rope":
        lead = (c["n"],) if c["n"] else ()
        s = dict(c=c, q=randn(*lead, c["T"], c["Hq"], c["d"]).to(TYPE[c["dtype"]]), k=randn(*lead, c["T"], c["Hkv"], c["d"]).to(TYPE[c["dtype"]]))
        if lead:  # [n, heads, T, d], as a projection of [n, T] tokens leaves them
            s["q"], s["k"] = s["q"].transpose(1, 2), s["k"].transpose(1, 2)
            first = torch.randint(0, c["far"], (c["n"], 1), device="cuda", generator=gen)
            s["pos"] = (first + torch.arange(c["T"], device="cuda")).int()
        else:  # packed: prompts of about a quarter of the rows, each from a position of its own
            per = c["T"] // 4 + 1
            first = torch.randint(0, c["far"], (4,), device="cuda", generator=gen)
            t = torch.arange(c["T"], device="cuda")
            s["pos"] = (first[t // per] + t % per).int()
        s["freq"], s["amp"] = _frequencies(c)
        if own:
            import block_sparse_attention_plan_gb300 as bsa
            s["rope"] = bsa.rope_create(c["rot"], base=c["base"], pairs=c["pairs"], scaling=c["scaling"], factor=c["factor"],
                                        original=c["original"])
        return s
    lens = _lens(c)
    if c["op"] == "prompt":
        T = sum(lens)
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        return dict(c=c, q=randn(T, c["Hq"], c["d"]).to(TYPE[c["dtype"]]), k=randn(T, c["Hkv"], c["d"]).to(TYPE[c["dtype"]]),
                    v=randn(T, c["Hkv"], c["d"]).to(TYPE[c["dtype"]]), offsets=torch.tensor(at, dtype=torch.int32, device="cuda"))
    s = _cache(gen, c, lens)
    cap = s["table"].shape[1] * c["page"]
    if c["op"] == "weigh":
        s["q"] = randn(c["n"], c["Hq"], c["nq"], c["d"]).to(torch.bfloat16)
        if c["bk"]:
            s["mask"] = _blocks(gen, c, lens)
        s["weights"] = torch.rand(c["n"], c["Hkv"], cap, device="cuda", generator=gen)
        # what the attention of these queries left: the logarithm of its sum, near that of as many standard scores
        n = torch.tensor(lens, dtype=torch.float32, device="cuda").view(-1, 1, 1)
        s["lse"] = torch.log(n) + 0.5 + 0.1 * randn(c["n"], c["Hq"], c["nq"])
        return s
    # weights as attention leaves them: a few large, most small, some nothing
    w = torch.exp(2.0 * randn(c["n"], c["Hkv"], cap))
    s["weights0"] = torch.where(torch.rand(w.shape, device="cuda", generator=gen) < 0.1, 0.0, w)
    s["weights"] = s["weights0"].clone()
    s["table0"], s["refs0"], s["lens0"] = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
    s["keep"] = torch.full((c["n"],), c["keep"], dtype=torch.int32, device="cuda")
    s["kept"] = torch.full((c["n"], c["Hkv"], min(cap, c["keep"])), -1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms

def _rotate(x, s, at, sign):
    """Rows x [..., heads, T, d] at angles [..., 1, T, rot / 2]."""
    c = s["c"]
    r = c["rot"]
    co, si = (torch.cos(at) * s["amp"]).float(), (torch.sin(at) * (s["amp"] * sign)).float()
    y = x.float()
    if c["pairs"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        z = torch.cat([a * co - b * si, b * co + a * si, y[..., r:]], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        z = torch.cat([torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2), y[..., r:]], -1)
    return z.to(x.dtype)


def _rope(s):
    at = (s["pos"].double().unsqueeze(-1) * s["freq"]).unsqueeze(-3 if s["c"]["n"] else -2)
    sign = -1.0 if s["c"]["inverse"] else 1.0
    return _rotate(s["q"], s, at, sign), _rotate(s["k"], s, at, sign)


def _prompt(s):
    """The prompts padded to the longest, their rows taken back out."""
    c, off = s["c"], s["offsets"].long()
    L, T, n, Hq, H, d = c["hi"], s["q"].shape[0], c["n"], c["Hq"], c["Hkv"], c["d"]
    j = torch.arange(L, device="cuda")
    rows = (off[:-1, None] + j).clamp(max=max(T - 1, 0))                                  # [n, L]
    q = s["q"][rows].float().view(n, L, H, Hq // H, d).permute(0, 2, 3, 1, 4)             # [n, H, g, L, d]
    k, v = (s[x][rows].float().transpose(1, 2).unsqueeze(2) for x in ("k", "v"))          # [n, H, 1, L, d]
    keep = (j < (off[1:] - off[:-1])[:, None]).view(n, 1, 1, 1, L)
    if c["causal"]:
        keep = keep & (j <= j[:, None])
    x = (q * d ** -0.5) @ k.transpose(-1, -2)
    x.masked_fill_(~keep, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e @ torch.where(keep[..., -1:, :].transpose(-1, -2), v, 0.0)) / total
    lse = (top + torch.log(total)).squeeze(-1)
    t = torch.arange(T, device="cuda")
    i = torch.searchsorted(off[1:], t, right=True)
    at = t - off[i]
    return o.to(s["q"].dtype)[i, :, :, at].reshape(T, Hq, d), lse[i, :, :, at].reshape(T, Hq)


def _at(x, *where):
    """x[where], moved as bytes."""
    return x.view(torch.uint8)[where].view(x.dtype)


def _weigh(s):
    c = s["c"]
    n, H, S, d, sb, nq, L = c["n"], c["Hkv"], c["page"], c["d"], c["sb"], c["nq"], s["weights"].shape[2]
    page = s["table"].long().clamp(min=0)
    k = _at(s["k"], page).view(n, -1, H, S // sb, sb, d).float() * s["ks"][page][..., None, None]
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(n, H, L, d)
    end, j = s["lens"].long().view(n, 1, 1, 1), torch.arange(L, device="cuda")
    keep = j < end
    if c["causal"]:
        keep = keep & (j <= end - nq + torch.arange(nq, device="cuda").view(-1, 1))
    if "mask" in s:
        m = s["mask"].bool().repeat_interleave(c["bk"], -1)[..., :L]
        m = torch.cat([m, m.new_zeros(n, c["Hq"], L - m.shape[-1])], -1)
        keep = keep & m.unsqueeze(2)
    x = (s["q"].float().view(n, H, -1, d) * d ** -0.5) @ k.transpose(-1, -2)
    p = torch.exp(x.view(n, c["Hq"], nq, L) - s["lse"].unsqueeze(-1))
    got = torch.where(keep, p, 0.0).view(n, H, -1, L).sum(2)
    end = end.squeeze(-1)
    w = torch.where(j >= end - c["fresh"], 0.0, s["weights"]) + got
    s["weights"].copy_(torch.where(j < end, w, s["weights"]))
    return s["weights"]


def _evict(s):
    c, table, w, lens = s["c"], s["table"], s["weights"], s["lens"]
    n, H, S, sb, L, W = c["n"], c["Hkv"], c["page"], c["sb"], w.shape[2], s["kept"].shape[2]
    k = torch.minimum(s["keep"], lens).long().view(n, 1, 1)
    end, j = lens.long().view(n, 1, 1), torch.arange(L, device="cuda")
    recent = k.clamp(max=c["recent"])
    sink = (k - recent).clamp(max=c["sink"])
    # sorted: what stays in any case, then by weight, the lowest index first, then what is no token
    rank = torch.where((j < sink) | (j >= end - recent), math.inf, w)
    rank = torch.where(j < end, rank, -1.0)
    order = torch.sort(rank, stable=True, dim=-1, descending=True).indices
    place = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    taken = torch.where(place < k, j, L + j)
    src = torch.sort(taken, -1).values[..., :W]                                          # ascending: the kept tokens first
    to = torch.arange(W, device="cuda")
    there = to < k                                                                       # [n, 1, W]
    src = torch.where(there, src, 0)
    s["kept"].copy_(torch.where(there, src, s["kept"].long()))
    w[..., :W] = torch.where(there, w.gather(2, src), w[..., :W])
    row, head = torch.arange(n, device="cuda").view(n, 1, 1), torch.arange(H, device="cuda").view(1, H, 1)
    cut = there & (end > s["keep"].view(n, 1, 1))
    bin_ = s["k"].shape[0] - 1
    page = table.long()[row, src // S].clamp(min=0)
    dest = torch.where(cut, table.long()[row, to // S], bin_).expand(n, H, W)
    put = to.expand(n, H, W)
    for x in ("k", "v"):
        old, was = _at(s[x], page, head, src % S), s[x + "s"][page, head, src % S // sb]
        # the largest scale of the tokens that come to lie in a block
        block = (to // sb).expand(n, H, W)
        now = torch.zeros(n, H, (W - 1) // sb + 1, device="cuda").scatter_reduce(2, block, torch.where(there, was, 0.0), "amax").gather(2, block)
        y = old.float() * torch.where(there, was / now, 0.0).unsqueeze(-1)
        y = y.to(CODE[E4M3]) if c["kind"] == E4M3 else y.round().to(torch.int8)
        s[x].view(torch.uint8)[dest, head, put % S] = y.view(torch.uint8)
        s[x + "s"][dest, head, put % S // sb] = now
    lens.copy_(torch.minimum(lens, s["keep"]))
    t = torch.arange(table.shape[1], device="cuda")
    gone = (t >= ((lens + S - 1) // S).view(n, 1)) & (table >= 0)
    s["refs"].sub_(torch.zeros(s["refs"].shape[0] + 1, dtype=torch.int32, device="cuda").scatter_add_(
        0, torch.where(gone, table.long(), s["refs"].shape[0]).flatten(), gone.flatten().int())[:-1])
    table.masked_fill_(gone, -1)


# --------------------------------------------------------------------------------------- run

def run(s):
    c = s["c"]
    if own:
        import block_sparse_attention_plan_gb300 as bsa
        if c["op"] == "rope":
            return bsa.rope(s["rope"], s["q"], s["k"], positions=s["pos"], inverse=c["inverse"])
        if c["op"] == "prompt":
            return bsa.prompt_attention(s["q"], s["k"], s["v"], s["offsets"], causal=c["causal"])
        if c["op"] == "weigh":
            bsa.cache_weigh(s["cache"], s["q"], s["lse"], s["weights"], mask=s.get("mask"), bk=c["bk"], causal=c["causal"], fresh=c["fresh"])
            return s["weights"]
    if c["op"] == "rope":
        return _rope(s)
    if c["op"] == "prompt":
        return _prompt(s)
    if c["op"] == "weigh":
        return _weigh(s)
    for x in ("table", "refs", "lens", "weights"):
        s[x].copy_(s[x + "0"])
    if own:
        bsa.cache_evict(s["cache"], s["weights"], s["keep"], sink=c["sink"], recent=c["recent"], kept=s["kept"])
    else:
        _evict(s)
    return dict(kept=s["kept"], weights=s["weights"], table=s["table"], lens=s["lens"], refs=s["refs"],
                k=s["k"][:-1], v=s["v"][:-1], ks=s["ks"][:-1], vs=s["vs"][:-1])


# ------------------------------------------------------------------------------------- exact

def _exact_rope(s):
    """Each pair as a complex number, times a power of e."""
    c, r = s["c"], s["c"]["rot"]
    base, f = c["base"], []
    for i in range(r // 2):
        x = base ** (-(2 * i) / r)
        amp = 1.0
        if c["scaling"] == "linear":
            x /= c["factor"]
        elif c["scaling"] == "base":
            x = (base * c["factor"] ** (r / max(r - 2, 1))) ** (-(2 * i) / r)
        elif c["scaling"] == "parts":
            turns = c["original"] * x / (2 * math.pi)
            stay = min(1.0, max(0.0, (turns - 1) / 31))
            x, amp = x * (stay + (1 - stay) / c["factor"]), 1 + 0.1 * math.log(c["factor"])
        f.append(x)
    turn = torch.polar(torch.full((1,), amp, dtype=torch.float64, device="cuda"),
                       s["pos"].double().unsqueeze(-1) * torch.tensor(f, dtype=torch.float64, device="cuda"))
    turn = (turn.conj() if c["inverse"] else turn).unsqueeze(1)  # [n or T, 1, (T,) r / 2]
    out = []
    for name in ("q", "k"):
        y = s[name].double().clone()
        first, second = (y[..., :r // 2], y[..., r // 2:r]) if c["pairs"] == "half" else (y[..., 0:r:2], y[..., 1:r:2])
        z = torch.complex(first.clone(), second.clone()) * turn
        first.copy_(z.real)
        second.copy_(z.imag)
        out.append(y)
    return tuple(out)


def _exact_prompt(s):
    c, off = s["c"], s["offsets"].tolist()
    T, Hq, d = s["q"].shape
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    for a, b in zip(off, off[1:]):
        for h in range(Hq):
            kv = h * c["Hkv"] // Hq
            for i in range(a, b, 2048):
                e = min(b, i + 2048)
                last = e if c["causal"] else b
                x = torch.einsum("td,jd->tj", s["q"][i:e, h].double(), s["k"][a:last, kv].double()) / math.sqrt(d)
                if c["causal"]:
                    x += torch.full_like(x, -math.inf).triu_(i - a + 1)
                z = torch.logsumexp(x, 1)
                o[i:e, h] = torch.softmax(x, 1) @ s["v"][a:last, kv].double()
                lse[i:e, h] = z
    return o, lse


def _exact_weigh(s):
    c = s["c"]
    out = s["weights"].double().clone()
    g, S, sb = c["Hq"] // c["Hkv"], c["page"], c["sb"]
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-n // S)].long()
        out[b, :, max(0, n - c["fresh"]):n] = 0
        j = torch.arange(n, device="cuda")
        for h in range(c["Hkv"]):
            keys = (_at(s["k"], pages, h).double().view(-1, sb, c["d"]) * s["ks"][pages, h].double().view(-1, 1, 1)).view(-1, c["d"])[:n]
            for x in range(h * g, (h + 1) * g):
                for i in range(c["nq"]):
                    p = torch.exp((keys @ s["q"][b, x, i].double()) / math.sqrt(c["d"]) - s["lse"][b, x, i].double())
                    if c["causal"]:
                        p = p * (j <= n - c["nq"] + i)
                    if "mask" in s:
                        p = p * (s["mask"][b, x, j // c["bk"]] != 0)
                    out[b, h, :n] += p
    return out


def _exact_evict(s):
    """Sequence by sequence: the indices that stay, and what lies there then."""
    c, S, sb = s["c"], s["c"]["page"], s["c"]["sb"]
    w = s["weights"].double().clone()
    pools = {x: s[x][:-1].double() for x in ("k", "v")} | {x: s[x][:-1].double() for x in ("ks", "vs")}
    for b, n in enumerate(s["lens"].tolist()):
        k = c["keep"]
        if n <= k:
            continue
        r = min(c["recent"], k)
        a = min(c["sink"], k - r)
        pages = s["table"][b].long()
        for h in range(c["Hkv"]):
            others = s["weights"][b, h, a:n - r]
            best = torch.sort(others, stable=True, dim=0, descending=True).indices[:k - r - a] + a
            stay = torch.cat([torch.arange(a, device="cuda"), torch.sort(best).values, torch.arange(n - r, n, device="cuda")])
            to = torch.arange(k, device="cuda")
            w[b, h, :k] = s["weights"][b, h, stay].double()
            for x in ("k", "v"):
                value = s[x + "s"][pages[stay // S], h, stay % S // sb].double()
                top = torch.stack([p.max() for p in value.split(sb)])
                y = _at(s[x], pages[stay // S], h, stay % S).double() * (value / top[to // sb]).unsqueeze(1)
                pools[x][pages[to // S], h, to % S] = _nearest(y, c["kind"])
                pools[x + "s"][pages[to // S], h, to % S // sb] = top[to // sb]
    return dict(kept=None, weights=w, table=None, lens=None, refs=None, k=pools["k"] if c["kind"] == E4M3 else None,
                v=pools["v"] if c["kind"] == E4M3 else None, ks=pools["ks"], vs=pools["vs"])


def _nearest(x, kind):
    """Nearest code value of x in 64 bits, ties to even."""
    if kind == INT8:
        return torch.round(x)
    a = x.abs()
    step = torch.exp2((torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 4).double())
    return torch.sign(x) * torch.round(a / step) * step


def exact(c, seed):
    if c["op"] == "weigh" and c["n"] * c["Hq"] * c["nq"] > 6000:
        return None
    s = prepare(c, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "weigh": _exact_weigh, "evict": _exact_evict}[c["op"]](s)
