"""What is measured of the paged cache's tables and of the attention of many rows over it.

  extend   pages, offsets, positions and slots of new tokens, from request lengths
  release  the pages of finished sequences, back to the free ones
  cross    attention of a sequence's tokens to all cached states of its encoder
  prefix   attention of one new token per sequence, groups of which share a cached prefix

`run` computes each in its plain form (`own` false: torch operations, sums in 32 bits) or by
the library's entry points (`own` true).  A cache page holds 128 tokens.  The record of (page,
KV head) is
  K codes [128, D/2] | V codes [128, D/2] | K scales [128, D/16] | V scales [128, D/16]
bytes: E2M1 codes, two a byte (the even element in the low nibble), and E4M3 scales of 16
elements each; the value is code * scale.  A query is quantized alike, with scale
s = E4M3(amax / 6) and code E2M1(x / s), both to nearest even and saturating, decided on fp32
quotients.  Token p of a sequence with table row t lies in slot 128 t[p / 128] + p % 128.
"""
import math
import random

import torch

own = False

PAGE = 128


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 sequences, one token each, some places of the batch idle
        dict(name="extend_step", op="extend", b=64, prompt=0, far=8192, start=False),
        # 48 prompts of uneven length admitted at once, positions counted from behind a prefix
        dict(name="extend_prompts", op="extend", b=48, prompt=131072, far=300, start=True),
        # a third of 64 sequences finished
        dict(name="release_step", op="release", b=64, far=8192, share=0.33),
        # every one of 8 long contexts given up
        dict(name="release_long", op="release", b=8, far=131072, share=1.0),
        # one new token per sequence, encoder states of uneven length, heads of 64: latency
        dict(name="cross_token", op="cross", b=64, n=1, ragged=False, h=16, hkv=16, d=64,
             longest=1500),
        # nine short pieces of a ragged batch, grouped heads, one encoder without states
        dict(name="cross_ragged", op="cross", b=9, n=37, ragged=True, h=32, hkv=8, d=128,
             longest=777),
        # about four latents of 4x28x56, texts of uneven length
        dict(name="cross_batch", op="cross", b=4, n=6272, ragged=True, h=12, hkv=12, d=128,
             longest=512),
        # one 21x30x52 latent, 12 heads, a full text of 512 tokens
        dict(name="cross_latent", op="cross", b=1, n=32760, ragged=False, h=12, hkv=12, d=128,
             longest=512),
        # a few samples of one prompt: latency
        dict(name="prefix_few", op="prefix", b=4, groups=1, h=32, hkv=8, d=128, prefix=2000,
             longest=200),
        # groups with prefixes of their own, one without any, heads of 64
        dict(name="prefix_groups", op="prefix", b=48, groups=4, h=16, hkv=2, d=64, prefix=16384,
             longest=1500),
        # a serving batch behind one system prompt
        dict(name="prefix_batch", op="prefix", b=64, groups=1, h=32, hkv=8, d=128, prefix=8192,
             longest=1024),
        # many samples over one long document
        dict(name="prefix_long", op="prefix", b=32, groups=1, h=64, hkv=8, d=128, prefix=131072,
             longest=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "release", "cross", "cross", "prefix", "prefix"])
    d = rng.choice([64, 128])
    if op == "extend":
        prompt = rng.choice([0, _log_int(rng, 20, 131072)])
        return dict(op=op, b=_log_int(rng, 1, 256), prompt=prompt, far=_log_int(rng, 100, 16384),
                    start=rng.random() < 0.5)
    if op == "release":
        return dict(op=op, b=_log_int(rng, 1, 256), far=_log_int(rng, 100, 16384),
                    share=rng.choice([0.1, 0.5, 1.0]))
    hkv = rng.randint(1, 12)
    h = hkv * rng.choice([1, 1, 2, 3, 4, 8])
    if op == "cross":
        b = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, 4096)
        # at most the largest listed case's rows and products
        top = 32760 * 12 // (b * h) * 512 // max(512, longest)
        return dict(op=op, b=b, n=_log_int(rng, 1, max(1, min(32760, top))),
                    ragged=rng.random() < 0.5, h=h, hkv=hkv, d=d, longest=longest)
    b = _log_int(rng, 1, 64)
    return dict(op=op, b=b, groups=rng.randint(1, min(4, b)), h=h, hkv=hkv, d=d,
                prefix=_log_int(rng, 1, 32 * 64 * 131072 // (64 * 96)),
                longest=_log_int(rng, 1, 2048))


def _spread(i, shift):
    """A fixed sequence of fractions, spread over [0, 1)."""
    return (i * 0.6180339887498949 + shift) % 1.0


def _growth(case):
    """(new tokens, tokens before them) of each sequence of an extend case."""
    b = case["b"]
    if case["prompt"]:
        share = [1.0 + _spread(i, 0.2) for i in range(b)]
        new = [int(case["prompt"] * s / sum(share)) for s in share]
        return [(n, 0 if i % 3 else int(case["far"] * _spread(i, 0.6))) for i, n in enumerate(new)]
    return [(0 if b >= 16 and i % 13 == 5 else 1, int(case["far"] * _spread(i, 0.11)))
            for i in range(b)]


def _finished(case):
    """(tokens, whether it is done) of each sequence of a release case."""
    b = case["b"]
    got = [(int(case["far"] * _spread(i, 0.37)), _spread(i, 0.9) < case["share"]) for i in range(b)]
    got[-1] = (case["far"], True)
    return got


def _lengths(b, top, empty):
    """Lengths spread over [1, top] with one at the top; where `empty`, some of many are 0."""
    got = [max(1, int(top * _spread(i, 0.37))) for i in range(b)]
    got[-1] = top
    if empty:
        got[1 % b] = 0
    return got


def _tokens(case):
    """Query tokens of each sequence of a cross case."""
    b, n = case["b"], case["n"]
    if not case["ragged"]:
        return [n] * b
    return [max(0, int(2 * n * _spread(i, 0.81))) for i in range(b - 1)] + [n]


def _encoder_lengths(case):
    return _lengths(case["b"], case["longest"], case["b"] >= 8)


def _groups(case):
    """(sequences, prefix length) of each group; the last of several shares nothing."""
    b, g = case["b"], case["groups"]
    cut = [b * i // g for i in range(g + 1)]
    top = case["prefix"]
    lens = [max(1, int(top * (1 - 0.2 * i))) for i in range(g)]
    if g > 2:
        lens[-1] = 0
    return [(cut[i + 1] - cut[i], lens[i]) for i in range(g)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    op = case["op"]
    if op == "extend":
        runs = _growth(case)
        tokens = sum(t for t, _ in runs)
        pages = sum(_pages(t + n) - _pages(n) for t, n in runs)
        return {"bytes": case["b"] * (16 + 4 * case["start"]) + pages * 8 + tokens * 12,
                "flops": tokens * 4}
    if op == "release":
        pages = sum(_pages(n) for n, done in _finished(case) if done)
        return {"bytes": case["b"] * 9 + pages * 8, "flops": pages}
    h, d = case["h"], case["d"]
    if op == "cross":
        lens, tokens = _encoder_lengths(case), _tokens(case)
        rows, keys = sum(tokens), sum(n for n, t in zip(lens, tokens) if t)
        pairs = sum(n * t for n, t in zip(lens, tokens))
    else:
        own_lens = _lengths(case["b"], case["longest"], case["b"] >= 16)
        rows, keys = case["b"], sum(own_lens) + sum(n for _, n in _groups(case))
        pairs = sum(own_lens) + sum(b * n for b, n in _groups(case))
    return {"bytes": keys * case["hkv"] * d * 9 / 8 + rows * h * (d * 4 + 4),
            "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------------------- NVFP4, plain

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x):
    """Packed codes (uint8 [..., n/2]) and E4M3 scales (float8 [..., n/16]) of x."""
    b = x.float().unflatten(-1, (-1, 16))
    # a tensor divisor: torch multiplies by the reciprocal of a Python number
    six = torch.full((), 6.0, device=x.device)
    s8 = (b.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    q = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    code = ((q > 0.25).byte() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) +
            (q > 5.0))
    code = (code + 8 * torch.signbit(b).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s8


def _unpack(packed, scales):
    """fp32 values of packed codes [..., n/2] and E4M3 scales [..., n/16]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    v = torch.stack((lut[(packed & 15).int()], lut[(packed >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _parts(pool, d):
    """Views K codes, V codes, K scales, V scales [pages, heads, 128, .] of a pool."""
    c, s = PAGE * d // 2, PAGE * d // 16
    kc, vc, ks, vs = pool.split([c, c, s, s], -1)
    f8 = torch.float8_e4m3fn
    return (kc.unflatten(-1, (PAGE, d // 2)), vc.unflatten(-1, (PAGE, d // 2)),
            ks.view(f8).unflatten(-1, (PAGE, d // 16)), vs.view(f8).unflatten(-1, (PAGE, d // 16)))


# ---------------------------------------------------------------------------- inputs

def _tables(gen, lens, spare=3):
    """A page table [rows, capacity] of shuffled pages for the given lengths, the pages that no
    row holds (int32, shuffled) and the number of all pages."""
    need = [_pages(n) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((len(lens), max(need + [0]) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, perm[at:].clone(), total


def _pool(gen, pages, hkv, d):
    """A pool as the append would have left it."""
    pool = torch.empty(pages, hkv, PAGE * d * 9 // 8, dtype=torch.uint8, device="cuda")
    for at in range(0, pages, 1024):
        kc, vc, ks, vs = _parts(pool[at:at + 1024], d)
        for codes, scales in ((kc, ks), (vc, vs)):
            x = torch.randn(*codes.shape[:-1], d, generator=gen, device="cuda")
            c, s = _quantize(x.to(torch.bfloat16))
            codes.copy_(c)
            scales.view(torch.uint8).copy_(s.view(torch.uint8))
    return pool


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _offsets(counts):
    got = [0]
    for n in counts:
        got.append(got[-1] + n)
    return _ints(got)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    st = dict(case)
    if case["op"] == "extend":
        runs = _growth(case)
        rng.shuffle(runs)
        lens = [n for _, n in runs]
        grown = [_pages(t + n) - _pages(n) for t, n in runs]
        st["table"], free, st["pages"] = _tables(gen, lens, spare=sum(grown) + 5)
        wide = max(_pages(t + n) for t, n in runs) + 1
        st["table"] = torch.nn.functional.pad(st["table"], (0, max(0, wide - st["table"].shape[1])),
                                              value=-1)
        st["free"] = torch.full((st["pages"],), -1, dtype=torch.int32, device="cuda")
        st["free"][:free.numel()] = free
        st["count"] = _ints([free.numel()])
        st["new"], st["lens"] = _ints([t for t, _ in runs]), _ints(lens)
        # rows of the step: a user's program sizes them by its batch, a few more than it needs
        st["tokens"] = sum(t for t, _ in runs) + (7 if case["prompt"] else 0)
        if not case["prompt"]:
            st["tokens"] = case["b"]
        st["start"] = None
        if case["start"]:
            st["start"] = _ints([rng.choice([0, 2000, 16384]) for _ in runs])
    elif case["op"] == "release":
        runs = _finished(case)
        rng.shuffle(runs)
        st["table"], free, st["pages"] = _tables(gen, [n for n, _ in runs], spare=11)
        st["free"] = torch.full((st["pages"],), -1, dtype=torch.int32, device="cuda")
        st["free"][:free.numel()] = free
        st["count"] = _ints([free.numel()])
        st["lens"] = _ints([n for n, _ in runs])
        st["done"] = _ints([f for _, f in runs], torch.bool)
    else:
        h, hkv, d = case["h"], case["hkv"], case["d"]
        if case["op"] == "cross":
            tokens, lens = _tokens(case), _encoder_lengths(case)
            rows = sum(tokens)
            st["cu"] = _offsets(tokens)
            st["table"], _, pages = _tables(gen, lens)
        else:
            rows, groups = case["b"], _groups(case)
            lens = _lengths(rows, case["longest"], rows >= 16)
            rng.shuffle(lens)
            prefixes = [n for _, n in groups]
            both, _, pages = _tables(gen, lens + prefixes)
            st["table"] = both[:rows, :_pages(max(lens)) + 1].contiguous()
            st["prefix_table"] = both[rows:, :max(1, _pages(max(prefixes)))].contiguous()
            st["prefix_lens"] = _ints(prefixes)
            st["cu"] = _offsets([b for b, _ in groups])
        st["lens"] = _ints(lens)
        st["pool"] = _pool(gen, pages, hkv, d)
        # the query part of a fused projection's output
        wide = torch.randn(rows, (h + 2 * hkv) * d, generator=gen, device="cuda")
        st["q"] = wide.to(torch.bfloat16)[:, :h * d].view(rows, h, d)
        st["scale"] = d ** -0.5
    return st


# ---------------------------------------------------------------------------- the plain forms

def _plain_extend(st):
    new, lens = st["new"].clamp(min=0).long(), st["lens"].clamp(min=0).long()
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    cu = torch.cat((zero, new.cumsum(0)))
    before, after = (lens + PAGE - 1) // PAGE, (lens + new + PAGE - 1) // PAGE
    first = torch.cat((zero, (after - before).cumsum(0)))  # new pages of the sequences before
    page = torch.arange(st["table"].shape[1], device="cuda")
    k = first[:-1, None] + page - before[:, None]
    fresh = (page >= before[:, None]) & (page < after[:, None])
    at = (st["count"].long() - 1 - k).clamp(0, st["pages"] - 1)
    st["table"].copy_(torch.where(fresh, st["free"][at], st["table"]))
    row = torch.arange(st["tokens"], device="cuda")
    seq = (torch.searchsorted(cu, row, right=True) - 1).clamp(max=st["b"] - 1)
    p = lens[seq] + row - cu[seq]
    live = row < cu[-1]
    p = torch.where(live, p, torch.zeros_like(p))
    slots = st["table"][seq, p // PAGE].long() * PAGE + p % PAGE
    positions = p if st["start"] is None else p + st["start"][seq]
    nothing = torch.full_like(p, -1)
    return dict(seq_lens=(lens + new).int(), free_count=(st["count"] - first[-1]).int(),
                cu_tokens=cu.int(), positions=torch.where(live, positions, nothing).int(),
                slots=torch.where(live, slots, nothing), page_table=st["table"])


def _plain_release(st):
    lens = torch.where(st["done"], st["lens"].clamp(min=0), torch.zeros_like(st["lens"])).long()
    pages = (lens + PAGE - 1) // PAGE
    first = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), pages.cumsum(0)))
    page = torch.arange(st["table"].shape[1], device="cuda")
    held = page < pages[:, None]
    at = (st["count"].long() + first[:-1, None] + page)[held]
    st["free"][at] = st["table"][held]
    return dict(seq_lens=torch.where(st["done"], torch.zeros_like(st["lens"]), st["lens"]),
                free_count=(st["count"] + first[-1]).int(), free_pages=st["free"])


def _rows_of(cu, rows):
    row = torch.arange(rows, device="cuda")
    return torch.searchsorted(cu.long(), row, right=True) - 1


def _attend(q, pool, table, lens, scale):
    """Sums of exp(S - m) V and of exp(S - m), and m, of q [R, Hkv, G, D] over the `lens` first
    keys of one table row (`lens` a tensor of one number)."""
    d = q.shape[-1]
    rec = pool[table.clamp(min=0).long()]
    kc, vc, ks, vs = (p.transpose(0, 1).flatten(1, 2) for p in _parts(rec, d))  # [Hkv, n, .]
    s = torch.einsum("rhgd,hnd->rhgn", q, _unpack(kc, ks)) * scale
    seen = torch.arange(s.shape[-1], device="cuda") < lens
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    return torch.einsum("rhgn,hnd->rhgd", p, _unpack(vc, vs)), p.sum(-1, keepdim=True), m


def _queries(st):
    hkv, h, d = st["hkv"], st["h"], st["d"]
    c, s = _quantize(st["q"])
    return _unpack(c, s).view(-1, hkv, h // hkv, d)


def _plain_cross(st):
    q = _queries(st)
    acc = torch.zeros_like(q)
    l, m = torch.zeros_like(q[..., :1]), torch.full_like(q[..., :1], -math.inf)
    counts = _tokens(st)  # a user's program knows its batch
    at = 0
    for i, n in enumerate(counts):
        r = slice(at, at + n)
        at += n
        acc[r], l[r], m[r] = _attend(q[r], st["pool"], st["table"][i], st["lens"][i], st["scale"])
    o = torch.where(l > 0, acc / l, torch.zeros_like(acc))
    return o.view(-1, st["h"], st["d"]).to(torch.bfloat16), (m + l.log()).view(-1, st["h"])


def _plain_prefix(st):
    b, h, hkv, d = (st[n] for n in ("b", "h", "hkv", "d"))
    q = _queries(st)
    acc = torch.zeros_like(q)
    l, m = torch.zeros_like(q[..., :1]), torch.full_like(q[..., :1], -math.inf)
    at = 0
    for i, (n, _) in enumerate(_groups(st)):
        r = slice(at, at + n)
        at += n
        acc[r], l[r], m[r] = _attend(q[r], st["pool"], st["prefix_table"][i], st["prefix_lens"][i],
                                     st["scale"])
    pages = st["pool"][st["table"].clamp(min=0).long()]  # own tokens [B, P, Hkv, record]
    kc, vc, ks, vs = (p.transpose(1, 2).flatten(2, 3) for p in _parts(pages, d))
    s = (q @ _unpack(kc, ks).mT) * st["scale"]
    seen = torch.arange(s.shape[-1], device="cuda") < st["lens"][:, None]
    s = torch.where(seen[:, None, None], s, torch.full_like(s, -math.inf))
    top = torch.maximum(m, s.amax(-1, keepdim=True))
    ref = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = torch.exp(s - ref)
    l = l * torch.exp(m - ref) + p.sum(-1, keepdim=True)
    acc = acc * torch.exp(m - ref) + p @ _unpack(vc, vs)
    o = torch.where(l > 0, acc / l, torch.zeros_like(acc))
    return o.view(b, h, d).to(torch.bfloat16), (top + l.log()).view(b, h)


# ---------------------------------------------------------------------------- one pass

def run(state):
    st, op = state, state["op"]
    if own:
        from nvfp4_fake_quant_gb300 import api
        if op == "extend":
            got = api.nvfp4_kv_extend(st["new"], st["lens"], st["table"], st["free"], st["count"],
                                      tokens=st["tokens"], start=st["start"])
            return got._asdict() | dict(page_table=st["table"])
        if op == "release":
            lens, count = api.nvfp4_kv_release(st["done"], st["lens"], st["table"], st["free"],
                                               st["count"])
            return dict(seq_lens=lens, free_count=count, free_pages=st["free"])
        if op == "cross":
            if "ws" not in st:  # kept by a serving loop, as the pool is
                st["ws"] = torch.empty(api.attn_qat_cross_workspace(
                    st["q"].shape[0], st["b"], st["h"], st["hkv"], st["d"], st["table"].shape[1]),
                    dtype=torch.uint8, device="cuda")
            return api.attn_qat_cross(st["q"], st["pool"], st["table"], st["lens"],
                                      cu_tokens=st["cu"] if st["ragged"] else None,
                                      scale=st["scale"], workspace=st["ws"])
        if "ws" not in st:
            st["ws"] = torch.empty(api.attn_qat_decode_prefix_workspace(
                st["b"], st["groups"], st["h"], st["hkv"], st["d"], st["table"].shape[1],
                st["prefix_table"].shape[1]), dtype=torch.uint8, device="cuda")
        return api.attn_qat_decode_prefix(st["q"], st["pool"], st["table"], st["lens"],
                                          st["prefix_table"], st["prefix_lens"],
                                          cu_seqs=st["cu"] if st["groups"] > 1 else None,
                                          scale=st["scale"], workspace=st["ws"])
    if op == "extend":
        return _plain_extend(st)
    if op == "release":
        return _plain_release(st)
    return _plain_cross(st) if op == "cross" else _plain_prefix(st)


# ---------------------------------------------------------------------------- in 64 bits

def _bytes64(codes, scales):
    """fp64 values of packed codes and E4M3 scale bytes, from the formats' bit fields."""
    c = torch.empty(*codes.shape, 2, dtype=torch.uint8, device=codes.device)
    c[..., 0], c[..., 1] = codes % 16, codes // 16
    e, m = (c // 2 % 4).double(), (c % 2).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2) * (1 - 2 * (c // 8).double())
    b = scales.view(torch.uint8)
    e, m = (b // 8 % 16).double(), (b % 8).double()
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)
    v = v.reshape(*codes.shape[:-1], -1, 16) * s[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _query64(x):
    """fp64 values of the quantized query: the scale's and the elements' roundings by distance to
    the nearest representable value, ties to the even, on the definition's fp32 quotients."""
    def nearest(v, grid):
        hi = torch.searchsorted(grid, v).clamp(max=len(grid) - 1)
        lo = (hi - 1).clamp(min=0)
        below, above = (v - grid[lo]).abs(), (grid[hi] - v).abs()
        pick_lo = (below < above) | ((below == above) & (lo % 2 == 0))
        return grid[torch.where(pick_lo, lo, hi)]

    e4m3 = [m * 2.0 ** -9 for m in range(8)]
    e4m3 += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    e4m3 = torch.tensor(e4m3, dtype=torch.float64, device=x.device)
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    blk = x.float().reshape(*x.shape[:-1], -1, 16)
    top = blk.abs().max(-1).values
    s = nearest((top / torch.tensor([6.0], device=x.device)).double(), e4m3)
    q = (blk.abs() / s.float()[..., None]).nan_to_num(0.0, posinf=0.0).double()
    return (torch.copysign(nearest(q, e2m1), blk.double()) * s[..., None]).reshape(x.shape)


def _exact_extend(st):
    """By the rules, one sequence and one token after another."""
    table, free = st["table"].cpu().tolist(), st["free"].tolist()
    left, cu, positions, slots, lens = int(st["count"]), [0], [], [], []
    start = [0] * st["b"] if st["start"] is None else st["start"].tolist()
    for i, (t, n) in enumerate(zip(st["new"].tolist(), st["lens"].tolist())):
        for p in range(n, n + t):
            if p % PAGE == 0:
                left -= 1
                table[i][p // PAGE] = free[left]
            positions.append(start[i] + p)
            slots.append(table[i][p // PAGE] * PAGE + p % PAGE)
        cu.append(cu[-1] + t)
        lens.append(n + t)
    rest = [-1] * (st["tokens"] - cu[-1])
    return dict(seq_lens=_ints(lens), free_count=_ints([left]), cu_tokens=_ints(cu),
                positions=_ints(positions + rest), slots=_ints(slots + rest, torch.int64),
                page_table=_ints(table))


def _exact_release(st):
    table, free, lens = st["table"].tolist(), st["free"].tolist(), st["lens"].tolist()
    count = int(st["count"])
    for i, done in enumerate(st["done"].tolist()):
        if done:
            for page in table[i][:_pages(lens[i])]:
                free[count] = page
                count += 1
            lens[i] = 0
    return dict(seq_lens=_ints(lens), free_count=_ints([count]), free_pages=_ints(free))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(st)
    if case["op"] == "release":
        return _exact_release(st)
    h, hkv, d = case["h"], case["hkv"], case["d"]
    q = _query64(st["q"]).view(-1, hkv, h // hkv, d)
    rows = q.shape[0]
    o = torch.zeros(rows, hkv, h // hkv, d, dtype=torch.float64, device="cuda")
    lse = torch.full(o.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")

    def keys(tables, lens, head):
        """fp64 K and V of one head: the first keys of each table row, one after another."""
        got = []
        for t, n in zip(tables, lens):
            if n == 0:
                continue
            rec = st["pool"][t[:_pages(n)].long(), head]
            kc, vc, ks, vs = (x[:, 0].reshape(-1, x.shape[-1])[:n] for x in _parts(rec[:, None], d))
            got.append((_bytes64(kc, ks), _bytes64(vc, vs)))
        return torch.cat([k for k, _ in got]), torch.cat([v for _, v in got])

    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    for head in range(hkv):
        if case["op"] == "cross":
            spans = [(range(cu[i], cu[i + 1]), [st["table"][i]], [lens[i]])
                     for i in range(case["b"])]
        else:
            shared = st["prefix_lens"].tolist()
            spans = [(range(r, r + 1), [st["prefix_table"][i], st["table"][r]], [shared[i], lens[r]])
                     for i in range(case["groups"]) for r in range(cu[i], cu[i + 1])]
        for span, tables, counts in spans:
            if not len(span) or not sum(counts):
                continue
            k, v = keys(tables, counts, head)
            for at in range(span.start, span.stop, 8192):
                r = slice(at, min(at + 8192, span.stop))
                s = q[r, head].flatten(0, 1) @ k.T * st["scale"]
                o[r, head] = (s.softmax(-1) @ v).view(-1, h // hkv, d)
                lse[r, head] = s.logsumexp(-1).view(-1, h // hkv)
    return o.view(rows, h, d), lse.view(rows, h)
