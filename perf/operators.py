"""Cases of the operators over a paged K/V cache held in 8 bits: appending tokens, attention of
single tokens and short drafts, chunked prefill over a block mask, and the page operations (fork,
grow, free, compact).

A cache is two pools of codes [pages, Hkv, page, d] (e4m3 or int8), an fp32 scale for each block of
`sb` tokens of a page and head, a page table [sequences, pages per sequence] (-1: none), a length per
sequence and a reference count per page; a value is code * scale.
"""
import math

import torch

own = False

E4M3, INT8 = "e4m3", "int8"
TOP = {E4M3: 448.0, INT8: 127.0}
CODE = {E4M3: torch.float8_e4m3fn, INT8: torch.int8}
MIN_EXP = -100  # smallest scale 2^-100


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a serving batch: a token per sequence, into partly filled blocks.
        dict(name="append_step", op="append", kind=E4M3, n=64, T=1, ragged=False, Hkv=8, d=128, page=64, sb=64, ctx=1500),
        # Prefill chunks of several prompts, of odd lengths, in 8-bit integers.
        dict(name="append_chunk", op="append", kind=INT8, n=6, T=4001, ragged=True, Hkv=16, d=64, page=32, sb=32, ctx=333),
        # One user, a short context: the latency of a call.
        dict(name="attn_one", op="attn", kind=E4M3, n=1, nq=1, Hq=32, Hkv=8, d=128, page=64, sb=64, lo=900, hi=901,
             causal=False, bk=0, topk=0),
        # A serving batch of mixed context lengths: the bulk of decoding.
        dict(name="attn_batch", op="attn", kind=E4M3, n=32, nq=1, Hq=32, Hkv=8, d=128, page=64, sb=64, lo=500, hi=32768,
             causal=False, bk=0, topk=0),
        # Draft tokens to be verified, causal among themselves; integer codes, small pages.
        dict(name="attn_draft", op="attn", kind=INT8, n=16, nq=5, Hq=32, Hkv=8, d=64, page=16, sb=16, lo=1000, hi=16000,
             causal=True, bk=0, topk=0),
        # Long contexts of which each head reads a sink, a window and its best blocks.
        dict(name="attn_blocks", op="attn", kind=E4M3, n=4, nq=1, Hq=32, Hkv=8, d=128, page=64, sb=64, lo=65000, hi=65536,
             causal=False, bk=64, topk=48),
        # A chunk of a long prompt over its prefix, each row of query blocks with its own key blocks.
        dict(name="prefill_chunk", op="prefill", kind=E4M3, n=1, Nq=1024, Nk=16384, short=0, Hq=32, Hkv=8, d=128, page=64,
             sb=64, bq=64, bk=64, window=16, topk=48, causal=True),
        # Two prompts of unequal length in one batch, heads without grouping, small blocks.
        dict(name="prefill_pair", op="prefill", kind=INT8, n=2, Nq=512, Nk=8192, short=700, Hq=16, Hkv=16, d=64, page=32,
             sb=32, bq=32, bk=32, window=32, topk=40, causal=True),
        # A step of a beam search over a few prompts: share, grow by a token, drop.
        dict(name="fork_few", op="fork", kind=E4M3, n=4, ways=4, Hkv=8, d=128, page=64, sb=64, lo=300, hi=2000, spare=200),
        # The same with many long sequences.
        dict(name="fork_many", op="fork", kind=E4M3, n=64, ways=4, Hkv=8, d=128, page=64, sb=64, lo=1000, hi=4000, spare=900),
        # A small pool after a few sequences ended.
        dict(name="compact_small", op="compact", kind=INT8, pages=600, live=0.5, Hkv=8, d=64, page=32, sb=32, seqs=16),
        # A large pool, a third of its pages free.
        dict(name="compact_large", op="compact", kind=E4M3, pages=8000, live=0.66, Hkv=8, d=128, page=64, sb=64, seqs=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attn", "attn", "attn", "prefill", "fork", "compact"])
    kind, d = rng.choice([E4M3, INT8]), rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    sb = rng.choice([s for s in (16, 32, 64, 128) if s <= page])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kind=kind, Hkv=Hkv, d=d, page=page, sb=sb)
    if op == "append":
        T = _log(rng, 1, 4000)
        return dict(c, n=_log(rng, 1, max(1, min(128, 24000 // T))), T=T, ragged=rng.random() < 0.5, ctx=_log(rng, 1, 3000))
    if op == "attn":
        n, g = _log(rng, 1, 64), rng.choice([1, 2, 4, 7, 8])
        hi = _log(rng, 70, max(100, min(60000, 1000000 // n)))
        bk = rng.choice([0, 0, 32, 64, 128])
        nq = rng.choice([1, 1, 1, 2, 3, 8])
        return dict(c, n=n, nq=nq, Hq=Hkv * g, lo=rng.randint(1, hi), hi=hi, causal=nq > 1, bk=bk,
                    topk=_log(rng, 1, 50) if bk else 0)
    if op == "prefill":
        b = rng.choice([32, 64, 128])
        Nq, n = 128 * rng.randint(1, 8), rng.randint(1, 2)
        Nk = Nq + 256 * rng.randint(0, 28)
        return dict(c, n=n, Nq=Nq, Nk=Nk, short=rng.randint(0, (Nk - Nq) // 2), Hq=Hkv * rng.choice([1, 2, 4]), bq=b, bk=b,
                    window=rng.randint(1, 16), topk=rng.randint(1, 48), causal=rng.random() < 0.5)
    if op == "fork":
        n, ways = _log(rng, 1, 64), rng.randint(1, 4)
        lo = rng.randint(1, 2000)
        return dict(c, n=n, ways=ways, lo=lo, hi=lo + rng.randint(1, 2000), spare=n * ways * 3 + rng.randint(0, 300))
    return dict(c, pages=_log(rng, 50, 8000), live=rng.uniform(0.2, 0.9), seqs=rng.randint(2, 64))


def _lens(c):
    """Lengths spread over [lo, hi]: the same for every seed."""
    return [c["lo"] + int((c["hi"] - c["lo"]) * ((i * 0.618034 + 0.9) % 1.0)) for i in range(c["n"])]


def _counts(c):
    return [max(1, c["T"] - (i * 377) % c["T"]) if c["ragged"] else c["T"] for i in range(c["n"])]


def _picked(c, n):
    """Key blocks that a group of heads reads of a sequence's n: a sink, a window of 16 and `topk` of the rest for each head."""
    rest = max(0, n - 17)
    g = c["Hq"] // c["Hkv"]
    k = min(c["topk"], rest)
    return min(n, 17), rest * (1 - (1 - k / rest) ** g) if rest else 0.0, k


def work(c):
    d, H = c["d"], c["Hkv"]
    if c["op"] == "append":
        t = sum(_counts(c))
        return {"bytes": 2 * t * H * d * (2 + 1) + 8 * t * H / c["sb"], "flops": 4 * t * H * d}
    if c["op"] == "attn":
        rows, keys, pairs = c["Hq"] * c["nq"], 0.0, 0.0
        for n in _lens(c):
            if c["bk"]:
                fixed, union, k = _picked(c, -(-n // c["bk"]))
                keys += min(n, (fixed + union) * c["bk"])
                pairs += rows * min(n, (fixed + k) * c["bk"])
            else:
                keys += n
                pairs += rows * n
        return {"bytes": keys * H * 2 * (d + 4 / c["sb"]) + c["n"] * rows * (4 * d + 4), "flops": 4 * d * pairs}
    if c["op"] == "prefill":
        lens = [c["Nk"] - i * c["short"] for i in range(c["n"])]
        share = min(1.0, (1 + c["window"] + c["topk"]) / (c["Nk"] / c["bk"]))
        return {"bytes": sum(lens) * H * 2 * d + c["n"] * c["Hq"] * c["Nq"] * (4 * d + 4),
                "flops": 4 * d * c["Hq"] * c["Nq"] * sum(lens) * share}
    per = 2 * H * (c["page"] * d + 4 * c["page"] // c["sb"])  # bytes of a page
    if c["op"] == "fork":
        lens = _lens(c)
        entries = sum(-(-n // c["page"]) for n in lens) * c["ways"]
        copies = sum(1 for n in lens if n % c["page"]) * c["ways"]
        return {"bytes": 2 * per * copies + entries * 4 * 4, "flops": 0}
    live = int(c["pages"] * c["live"])
    return {"bytes": 2 * per * live * (1 - c["live"]) + c["pages"] * 4 * 3, "flops": 0}


# ------------------------------------------------------------------------------------ inputs

def _scale_for(amax, kind):
    """Smallest power of two (at least 2^MIN_EXP) that takes |x| <= amax into the codes' range."""
    # amax = m 2^e with m in [0.5, 1); the codes' largest value is t 2^u likewise: amax <= 448 2^k where e - u <= k, or
    # one more where m > t
    m, e = torch.frexp(amax)
    t, u = math.frexp(TOP[kind])
    k = torch.where(amax > 0, e - u + (m > t).int(), MIN_EXP).clamp(min=MIN_EXP)
    return ((k + 127) << 23).view(torch.float32)  # 2^k, by its bits


def _encode(x, kind):
    """Nearest codes of x, ties to even, saturated."""
    x = x.clamp(-TOP[kind], TOP[kind])
    return (x if kind == E4M3 else x.round()).to(CODE[kind])


def _fill(gen, pages, c, spread=True):
    """Codes and scales of pages of N(0, 1) tokens, some heads and blocks of other magnitudes. One page more than asked
    for: the plain form writes there what goes nowhere."""
    H, S, d, sb = c["Hkv"], c["page"], c["d"], c["sb"]
    codes = torch.empty(pages + 1, H, S // sb, sb, d, dtype=CODE[c["kind"]], device="cuda")
    scales = torch.empty(pages + 1, H, S // sb, device="cuda")
    step = max(1, (1 << 26) // (H * S * d))
    for a in range(0, pages + 1, step):
        b = min(pages + 1, a + step)
        x = torch.randn(b - a, H, S // sb, sb, d, device="cuda", generator=gen)
        if spread:
            x *= torch.exp2(torch.rand(b - a, H, S // sb, 1, 1, device="cuda", generator=gen) * 2 - 1)
        s = _scale_for(x.abs().amax((-1, -2)), c["kind"])
        scales[a:b] = s
        codes[a:b] = _encode(x / s[..., None, None], c["kind"])
    return codes.view(pages + 1, H, S, d), scales


def _cache(gen, c, lens, rows, width, spare, extra=0):
    """A cache of sequences in shuffled pages, with `spare` free ones: its tensors, and the framework's handle of them."""
    S = c["page"]
    held = [-(-n // S) for n in lens]
    pages = sum(held) + spare
    perm = torch.randperm(pages, device="cuda", generator=gen).int()
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = perm[at:at + h]
        at += h
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[perm[:at].long()] = 1
    k, ks = _fill(gen, pages, c)
    v, vs = _fill(gen, pages, c)
    ln = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ln[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    return _handle(dict(c=c, k=k, v=v, ks=ks, vs=vs, table=table, lens=ln, refs=refs))


def _handle(s):
    if own:
        import block_sparse_attention_plan_gb300 as bsa
        s["cache"] = bsa.Cache(s["k"][:-1], s["v"][:-1], s["ks"][:-1], s["vs"][:-1], s["table"], s["lens"], s["refs"])
    return s


def _top_blocks(gen, shape, n, window, topk):
    """Per row: block 0, the last `window` blocks of its n, and `topk` of the others."""
    score = torch.rand(*shape, device="cuda", generator=gen)
    j = torch.arange(shape[-1], device="cuda")
    n = n.unsqueeze(-1)
    score = torch.where((j >= 1) & (j < n - window), score, -1.0)
    best = torch.sort(score, -1, descending=True).values[..., min(topk, shape[-1]) - 1:min(topk, shape[-1])]
    return ((j == 0) | ((j >= n - window) & (j < n)) | ((score >= best) & (score >= 0))).to(torch.uint8)


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(torch.bfloat16)
    S, H, d = c["page"], c["Hkv"], c["d"]
    if c["op"] == "append":
        counts = _counts(c)
        lens = [c["ctx"] + (i * 37) % 100 + t for i, t in enumerate(counts)]  # room is there already
        s = _cache(gen, c, lens, c["n"], -(-max(lens) // S), 2)
        amp = torch.exp2(torch.rand(c["n"], H, 1, 1, device="cuda", generator=gen) * 4 - 2)
        s["new_k"] = (torch.randn(c["n"], H, c["T"], d, device="cuda", generator=gen) * amp).to(torch.bfloat16)
        s["new_v"] = randn(c["n"], H, c["T"], d)
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        return s
    if c["op"] == "attn":
        lens = _lens(c)
        s = _cache(gen, c, lens, c["n"], -(-max(lens) // S), 2)
        s["q"] = randn(c["n"], c["Hq"], c["nq"], d)
        if c["bk"]:
            blocks = -(-max(lens) // c["bk"])
            n = torch.tensor([-(-x // c["bk"]) for x in lens], device="cuda").view(-1, 1).expand(-1, c["Hq"])
            s["mask"] = _top_blocks(gen, (c["n"], c["Hq"], blocks), n, 16, c["topk"])
        return s
    if c["op"] == "prefill":
        lens = [c["Nk"] - i * c["short"] for i in range(c["n"])]
        s = _cache(gen, c, lens, c["n"], -(-c["Nk"] // S), 2)
        s["q"] = randn(c["n"], c["Hq"], c["Nq"], d)
        q0 = (torch.tensor(lens, device="cuda") - c["Nq"]).view(-1, 1) + torch.arange(0, c["Nq"], c["bq"], device="cuda")
        n = ((q0 + c["bq"] - 1) // c["bk"] + 1).unsqueeze(1).expand(-1, c["Hq"], -1)
        s["mask"] = _top_blocks(gen, (c["n"], c["Hq"], c["Nq"] // c["bq"], c["Nk"] // c["bk"]), n, c["window"], c["topk"])
        return s
    if c["op"] == "fork":
        lens = _lens(c)
        m = c["n"] * c["ways"]
        s = _cache(gen, c, lens, c["n"] + m, -(-(max(lens) + 1) // S), c["spare"])
        s["src"] = torch.arange(c["n"], dtype=torch.int32, device="cuda").repeat_interleave(c["ways"])
        s["dst"] = torch.arange(c["n"], c["n"] + m, dtype=torch.int32, device="cuda")
        s["grown"] = s["lens"][s["src"].long()] + 1
        return s
    held = int(c["pages"] * c["live"])
    lens = [((held * (i + 1)) // c["seqs"] - (held * i) // c["seqs"]) * S for i in range(c["seqs"])]
    s = _cache(gen, c, lens, c["seqs"], -(-max(max(lens), 1) // S), c["pages"] - held)
    s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
    return s


# ------------------------------------------------------------------------------- plain forms

def _append(pool, scales, s, new):
    c = s["c"]
    H, S, d, sb, T, n = c["Hkv"], c["page"], c["d"], c["sb"], c["T"], c["n"]
    count = s["counts"].long().view(n, 1)
    end = s["lens"].long().view(n, 1)
    pos = end - count
    block = pos // sb + torch.arange((T - 1) // sb + 2, device="cuda")              # [n, nb]
    touched = block * sb < end
    page = s["table"].long().gather(1, (block * sb // S).clamp(max=s["table"].shape[1] - 1))
    page = torch.where(touched, page, pool.shape[0] - 1)
    sub = block * sb % S // sb
    tok = (block * sb).unsqueeze(-1) + torch.arange(sb, device="cuda")              # [n, nb, sb]
    is_new = (tok >= pos.unsqueeze(-1)) & (tok < end.unsqueeze(-1))
    is_old = tok < pos.unsqueeze(-1)
    at = (tok - pos.unsqueeze(-1)).clamp(0, T - 1).view(n, 1, -1, 1).expand(-1, H, -1, d)
    x = new.gather(2, at).view(n, H, -1, sb, d).transpose(1, 2).float()            # [n, nb, H, sb, d]
    blocks = pool.view(-1, H, S // sb, sb, d)
    old, was = _at(blocks, page, slice(None), sub), scales[page, :, sub]
    fresh = is_new[:, :, None, :, None]
    need = _scale_for(torch.where(fresh, x.abs(), 0.0).amax((-1, -2)), c["kind"])
    now = torch.where(is_old.any(-1).unsqueeze(-1), torch.maximum(need, was), need)
    moved = _encode(old.float() * (was / now)[..., None, None], c["kind"])
    keep = is_old[:, :, None, :, None]
    out = torch.where(fresh, _encode(x / now[..., None, None], c["kind"]).view(torch.uint8),
                      torch.where(keep, moved.view(torch.uint8), old.view(torch.uint8)))
    blocks.view(torch.uint8)[page, :, sub] = out
    scales[page, :, sub] = now


def _at(x, *where):
    """x[where], moved as bytes."""
    return x.view(torch.uint8)[where].view(x.dtype)


def _values(pool, scales, s, n, keys, dtype):
    """[n, Hkv, keys, d]: the values of the sequences' first `keys` tokens."""
    c = s["c"]
    H, S, d, sb = c["Hkv"], c["page"], c["d"], c["sb"]
    page = s["table"][:n, :-(-keys // S)].long().clamp(min=0)
    x = _at(pool, page).view(n, -1, H, S // sb, sb, d).to(dtype) * scales[page].to(dtype)[..., None, None]
    return x.permute(0, 2, 1, 3, 4, 5).reshape(n, H, -1, d)[:, :, :keys]


def _attend(q, k, v, keep, dtype):
    """Softmax attention; keep [n, Hq, nq, keys]; a row that keeps nothing gives 0 and -inf."""
    n, Hq, nq, d = q.shape
    H = k.shape[1]
    x = q.to(dtype).view(n, H, -1, d) @ k.transpose(-1, -2) * d ** -0.5
    x = torch.where(keep.reshape(x.shape), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return o.view(n, Hq, nq, d), lse.view(n, Hq, nq)


def _keep(s):
    c = s["c"]
    n, Hq, nq = s["q"].shape[:3]
    end = s["lens"][:n].long().view(n, 1, 1, 1)
    keys = s["mask"].shape[-1] * c["bk"] if "mask" in s else c["hi"]
    j = torch.arange(keys, device="cuda")
    keep = j < end
    if c["causal"]:
        keep = keep & (j <= end - nq + torch.arange(nq, device="cuda").view(-1, 1))
    if "mask" in s:
        m = s["mask"].bool()
        m = m.unsqueeze(2) if m.dim() == 3 else m.repeat_interleave(c["bq"], 2)
        keep = keep & m.repeat_interleave(c["bk"], -1)
    top = min(keys, s["table"].shape[1] * c["page"])  # a last block past every page holds no key
    return keep.expand(n, Hq, nq, keys)[..., :top], top


def _fork(s):
    """Shares the pages of src with dst, grows dst by a token each (a page of its own where the last one is shared and
    partly filled, the lowest free page first), and returns the tables in between; then frees dst."""
    c, table, lens, refs = s["c"], s["table"], s["lens"], s["refs"]
    S, src, dst = c["page"], s["src"].long(), s["dst"].long()
    table[dst], lens[dst] = table[src], lens[src]
    pages = table[dst]
    refs += torch.bincount(pages.flatten().long() + 1, minlength=refs.shape[0] + 1)[1:].int()
    have, want = lens[dst].long(), s["grown"].long()
    last = have % S != 0                                       # the new token goes into the last page
    page = table[dst, ((have - 1).clamp(min=0) // S)].long()
    same = (page.view(-1, 1) == page) & last & last.view(-1, 1)
    rank = same.tril(-1).sum(1)
    copied = last & (refs[page] - rank > 1)
    need = copied | ~last
    free = torch.sort((refs > 0).to(torch.uint8), stable=True).indices
    got = free[(need.cumsum(0) - 1).clamp(min=0)]
    table[dst, (want - 1) // S] = torch.where(need, got, page).int()
    bin_ = s["k"].shape[0] - 1
    to = torch.where(copied, got, bin_)
    for name in ("k", "v"):
        s[name].view(torch.uint8)[to] = s[name].view(torch.uint8)[page]
        s[name + "s"][to] = s[name + "s"][page]
    refs.index_add_(0, page, -copied.int())
    refs.index_add_(0, got, need.int())
    lens[dst] = s["grown"]
    out = dict(table=table.clone(), lens=lens.clone(), refs=refs.clone())
    pages = table[dst]
    refs -= torch.bincount(pages.flatten().long() + 1, minlength=refs.shape[0] + 1)[1:].int()
    table[dst], lens[dst] = -1, 0
    return out


def _compact(s):
    table, refs = s["table"], s["refs"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(refs.shape[0], device="cuda")
    moved = (live & (at >= count)).nonzero().view(-1)
    hole = (~live & (at < count)).nonzero().view(-1)
    to = at.clone()
    to[moved] = hole
    for name in ("k", "v"):
        s[name].view(torch.uint8)[hole] = s[name].view(torch.uint8)[moved]
        s[name + "s"][hole] = s[name + "s"][moved]
    refs[hole] = refs[moved]
    refs[moved] = 0
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)], -1))


def _pools(s):
    return dict(k=s["k"][:-1], v=s["v"][:-1], ks=s["ks"][:-1], vs=s["vs"][:-1])


# --------------------------------------------------------------------------------------- run

def run(s):
    c = s["c"]
    if own:
        import block_sparse_attention_plan_gb300 as bsa
        cache = s["cache"]
        if c["op"] == "append":
            bsa.cache_append(cache, s["new_k"], s["new_v"], counts=s["counts"])
            return _pools(s)
        if c["op"] == "attn":
            return bsa.cache_attention(cache, s["q"], mask=s.get("mask"), bk=c["bk"], causal=c["causal"])
        if c["op"] == "prefill":
            plan = bsa.plan(s["mask"], c["bq"], c["bk"], c["Hq"] // c["Hkv"], flags=bsa.PLAN_NO_UNION)
            return bsa.cache_forward(plan, cache, s["q"], causal=c["causal"])
        if c["op"] == "fork":
            bsa.cache_fork(cache, s["src"], s["dst"])
            bsa.cache_resize(cache, s["grown"], seqs=s["dst"])
            out = dict(table=s["table"].clone(), lens=s["lens"].clone(), refs=s["refs"].clone())
            bsa.cache_free(cache, seqs=s["dst"])
            return dict(between=out, table=s["table"], lens=s["lens"], refs=s["refs"], **_pools(s))
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        bsa.cache_compact(cache)
        return dict(table=s["table"], refs=s["refs"], **_pools(s))
    if c["op"] == "append":
        _append(s["k"], s["ks"], s, s["new_k"])
        _append(s["v"], s["vs"], s, s["new_v"])
        return _pools(s)
    if c["op"] in ("attn", "prefill"):
        keep, keys = _keep(s)
        n = c["n"]
        o, lse = _attend(s["q"], _values(s["k"], s["ks"], s, n, keys, torch.float32),
                         _values(s["v"], s["vs"], s, n, keys, torch.float32), keep, torch.float32)
        return o.to(torch.bfloat16), lse
    if c["op"] == "fork":
        out = _fork(s)
        return dict(between=out, table=s["table"], lens=s["lens"], refs=s["refs"], **_pools(s))
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    _compact(s)
    return dict(table=s["table"], refs=s["refs"], **_pools(s))


# ------------------------------------------------------------------------------------- exact

def _nearest(x, kind):
    """Nearest code value of x in 64 bits, ties to even, saturated."""
    if kind == INT8:
        return torch.round(x).clamp(-127, 127)
    a = x.abs().clamp(max=448.0)
    spacing = torch.tensor([2.0 ** (e - 4) for e in range(-5, 10)], dtype=torch.float64, device=x.device)  # of [2^(e-1), 2^e)
    step = spacing[(torch.frexp(a.clamp(min=2.0 ** -6)).exponent + 5).long()]
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_append(s, name, new):
    c = s["c"]
    S, sb, top = c["page"], c["sb"], TOP[c["kind"]]
    codes, scales = s[name][:-1].double(), s[name + "s"][:-1].double()
    table, lens, counts = s["table"].tolist(), s["lens"].tolist(), s["counts"].tolist()
    powers = torch.tensor([2.0 ** e for e in range(MIN_EXP, 121)], dtype=torch.float64, device="cuda")
    for i in range(c["n"]):
        a = lens[i] - counts[i]
        while a < lens[i]:
            b = min(lens[i], (a // sb + 1) * sb)
            p, r = table[i][a // S], a % S
            x = new[i, :, a - (lens[i] - counts[i]):b - (lens[i] - counts[i])].double()   # [H, tokens, d]
            u = r // sb
            big = x.abs().amax((1, 2))
            sc = powers[torch.searchsorted(powers * top, big)]  # the first that reaches the largest value
            first = r - r % sb
            if r > first:
                was = scales[p, :, u]
                sc = torch.maximum(sc, was)
                codes[p, :, first:r] = _nearest(codes[p, :, first:r] * (was / sc).view(-1, 1, 1), c["kind"])
            codes[p, :, r:r + b - a] = _nearest(x / sc.view(-1, 1, 1), c["kind"])
            scales[p, :, u] = sc
            a = b
    return (codes if c["kind"] == E4M3 else None), scales


def exact(c, seed):
    if c["op"] in ("fork", "compact"):
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        if sum(_counts(c)) // c["sb"] + c["n"] > 4000:
            return None
        k, ks = _exact_append(s, "k", s["new_k"])
        v, vs = _exact_append(s, "v", s["new_v"])
        return dict(k=k, v=v, ks=ks, vs=vs)
    # row by row of the batch: scores, their log of the sum of exponentials, the weighted mean of the values
    n, Hq, nq, d = s["q"].shape
    g = Hq // c["Hkv"]
    o = torch.zeros(n, Hq, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    S, sb = c["page"], c["sb"]
    for b in range(n):
        L = int(s["lens"][b])
        pages = s["table"][b, :-(-L // S)].long()
        for h in range(c["Hkv"]):
            w = [(_at(s[x], pages, h).double().view(-1, S // sb, sb, d) * s[x + "s"][pages, h].double()[..., None, None]).view(-1, d)[:L]
                 for x in ("k", "v")]
            hs = slice(h * g, (h + 1) * g)
            x = torch.einsum("gqd,kd->gqk", s["q"][b, hs].double(), w[0]) / math.sqrt(d)
            j, i = torch.arange(L, device="cuda"), torch.arange(nq, device="cuda").view(-1, 1)
            drop = (j > L - nq + i) if c["causal"] else torch.zeros(nq, L, dtype=torch.bool, device="cuda")
            drop = drop.expand(g, nq, L)
            if "mask" in s:
                m = s["mask"][b, hs]
                m = m.unsqueeze(1).expand(-1, nq, -1) if m.dim() == 2 else m[:, i.view(-1) // c["bq"]]
                drop = drop | (m[..., j // c["bk"]] == 0)
            x = x.masked_fill(drop, -math.inf)
            z = torch.logsumexp(x, -1)
            some = z > -math.inf
            p = torch.exp(x - torch.where(some, z, 0.0).unsqueeze(-1))
            o[b, hs], lse[b, hs] = torch.einsum("gqk,kd->gqd", p, w[1]), z
    return o, lse
