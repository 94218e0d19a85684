"""What is measured of the single-token serving operators and of the rotary positions.

  rope     rotary positions of Q and K (forward, and the gradient's rotation back)
  append   new tokens' K and V quantized to NVFP4 into the pages of a cache
  decode   attention of one new token per sequence over the paged NVFP4 cache
  linear   the NVFP4 linear of a few rows on weights packed once

`run` computes each in its plain form (`own` false: torch operations in 32 bits, angles in
64) or by the library's entry points (`own` true).  NVFP4 here: blocks of 16 elements, scale
s = E4M3(amax * g / 6), code E2M1(x * g / s), both to nearest even and saturating, decided on
fp32 products and quotients; the value is code * s / g.

A cache page holds 128 tokens.  The record of (page, KV head) is
  K codes [128, D/2] | V codes [128, D/2] | K scales [128, D/16] | V scales [128, D/16]
bytes, two codes a byte (the even element in the low nibble), scales as E4M3.  Weights: codes
[N, K/2] and scales in the 128x4 tiled layout that nvfp4_quantize_tiled writes.
"""
import math
import random

import torch

own = False

PAGE = 128


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one step of a 64-sequence batch, grouped heads, far positions of a context extended
        # by parts (slow frequencies interpolated): latency counts
        dict(name="rope_step", op="rope", t=64, hq=32, hk=8, d=128, rot=128, interleaved=False,
             axes=1, far=131072, factor=16.0, inverse=False),
        # Q and K of one 16x28x56 latent, 12 heads, three axes of positions, adjacent pairs
        dict(name="rope_latent", op="rope", t=25088, hq=12, hk=12, d=128, rot=128,
             interleaved=True, axes=3, far=56, factor=1.0, inverse=False),
        # the gradient of the rotation at the 21x30x52 latent's token count, half of each head
        # rotated, half layout
        dict(name="rope_part_bwd", op="rope", t=32760, hq=12, hk=12, d=128, rot=64,
             interleaved=False, axes=1, far=32760, factor=1.0, inverse=True),
        # one new token of each of 64 sequences, two of them empty places of a padded batch
        dict(name="append_step", op="append", b=64, hkv=8, d=128, prompt=0, far=8192),
        # five prompts of uneven length written at once, 12 heads
        dict(name="append_prompt", op="append", b=5, hkv=12, d=128, prompt=25088, far=0),
        # one short sequence: latency
        dict(name="decode_short", op="decode", b=1, h=12, hkv=12, d=128, longest=777, window=0,
             sinks=0),
        # a serving batch of uneven lengths, four query heads a KV head, two empty places
        dict(name="decode_batch", op="decode", b=64, h=32, hkv=8, d=128, longest=8192, window=0,
             sinks=0),
        # sliding window with a few first tokens that stay visible, heads of 64
        dict(name="decode_window", op="decode", b=32, h=16, hkv=2, d=64, longest=32760,
             window=4096, sinks=4),
        # few long contexts, eight query heads a KV head
        dict(name="decode_long", op="decode", b=8, h=64, hkv=8, d=128, longest=131072, window=0,
             sinks=0),
        # fused QKV projection (3 x 1536) of one token: latency
        dict(name="linear_one", op="linear", m=1, n=4608, k=1536, bias=True),
        # FFN down-projection of five tokens
        dict(name="linear_down", op="linear", m=5, n=1536, k=8960, bias=True),
        # a large layer at a batch of 32
        dict(name="linear_large", op="linear", m=32, n=28672, k=8192, bias=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "linear"])
    d = rng.choice([64, 128])
    if op == "rope":
        axes = rng.choice([1, 1, 3])
        hk = rng.randint(1, 12)
        return dict(op=op, t=_log_int(rng, 1, 32760), hq=hk * rng.choice([1, 1, 2]), hk=hk, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4 * 3]), interleaved=rng.random() < 0.5,
                    axes=axes, far=_log_int(rng, 64, 1 << 20) if axes == 1 else 56,
                    factor=rng.choice([1.0, 4.0, 16.0]) if axes == 1 else 1.0,
                    inverse=rng.random() < 0.5)
    if op == "append":
        if rng.random() < 0.5:
            return dict(op=op, b=_log_int(rng, 1, 256), hkv=rng.randint(1, 12), d=d, prompt=0,
                        far=_log_int(rng, 200, 32760))
        return dict(op=op, b=rng.randint(1, 9), hkv=rng.randint(1, 12), d=d,
                    prompt=_log_int(rng, 20, 25088), far=rng.choice([0, 300]))
    if op == "decode":
        b, hkv = _log_int(rng, 1, 64), rng.randint(1, 12)
        # at most the largest listed case's keys
        longest = _log_int(rng, 1, max(2, min(131072, 8 * 8 * 131072 // (2 * b * hkv))))
        window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        return dict(op=op, b=b, h=hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), hkv=hkv, d=d,
                    longest=longest, window=window, sinks=rng.choice([0, 1, 4, 130]))
    return dict(op=op, m=_log_int(rng, 1, 64), n=16 * _log_int(rng, 4, 1024),
                k=64 * _log_int(rng, 2, 128), bias=rng.random() < 0.5)


def _lengths(case):
    """Sequence lengths of a decode case, spread over [1, longest] with one at the longest;
    from 16 sequences on two places are empty (a padded batch)."""
    b, top = case["b"], case["longest"]
    got = [max(1, int(top * ((i * 0.6180339887498949 + 0.37) % 1.0))) for i in range(b)]
    got[-1] = top
    if b >= 16:
        got[1] = got[b // 2] = 0
    return got


def _prompts(case):
    """(new tokens, tokens before them) of each sequence of an append case."""
    b = case["b"]
    if case["prompt"]:
        share = [1.0 + (i * 0.6180339887498949) % 1.0 for i in range(b)]
        new = [max(1, int(case["prompt"] * s / sum(share))) for s in share]
        return [(n, (i * 61) % 200 if case["far"] else 0) for i, n in enumerate(new)]
    got = [(1, int(case["far"] * ((i * 0.6180339887498949 + 0.11) % 1.0))) for i in range(b)]
    if b >= 16:
        got[1] = got[b // 2] = (1, -1)  # length 0: nothing is written
    return got


def _visible(case):
    w, s = case["window"], case["sinks"]
    if not w:
        return sum(_lengths(case))
    return sum(min(n, min(n, w) + min(s, max(0, n - w))) for n in _lengths(case))


def work(case):
    if case["op"] == "rope":
        n = case["t"] * (case["hq"] + case["hk"])
        return {"bytes": n * case["d"] * 4 + case["t"] * case["axes"] * 4,
                "flops": n * case["rot"] * 3}
    if case["op"] == "append":
        n = sum(t for t, before in _prompts(case) if before >= 0) * case["hkv"] * case["d"] * 2
        return {"bytes": n * 2 + n * 9 / 16, "flops": n * 4}
    if case["op"] == "decode":
        keys = _visible(case)
        return {"bytes": keys * case["hkv"] * case["d"] * 9 / 8 + case["b"] * case["h"] *
                (case["d"] * 4 + 4), "flops": 4 * keys * case["h"] * case["d"]}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": n * k * 9 / 16 + (m * k + m * n) * 2 + (n * 2 if case["bias"] else 0),
            "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------- NVFP4, plain

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x, g=None):
    """Codes (uint8 [..., n], sign << 3 | index) and E4M3 scales (float8 [..., n/16]) of x."""
    b = x.float().unflatten(-1, (-1, 16))
    bg = b if g is None else b * g
    # a tensor divisor: torch multiplies by the reciprocal of a Python number
    six = torch.full((), 6.0, device=x.device)
    s8 = (bg.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    q = torch.where(s > 0, bg.abs() / s, torch.zeros_like(bg))
    code = ((q > 0.25).byte() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) +
            (q > 5.0))
    return (code + 8 * torch.signbit(b).byte()).flatten(-2), s8


def _pack(codes):
    return codes[..., 0::2] + 16 * codes[..., 1::2]


def _unpack(packed, scales):
    """fp32 values of packed codes [..., n/2] and E4M3 scales [..., n/16]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    v = torch.stack((lut[(packed & 15).int()], lut[(packed >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _tile_scales(s8):
    """[rows, blocks] scales in the 128x4 tiled layout (bytes)."""
    r, c = s8.shape
    p = torch.zeros((r + 127) // 128 * 128, (c + 3) // 4 * 4, dtype=torch.uint8, device=s8.device)
    p[:r, :c] = s8.view(torch.uint8)
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untile_scales(flat, r, c):
    p = flat.view((r + 127) // 128, (c + 3) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return p.reshape((r + 127) // 128 * 128, -1)[:r, :c].view(torch.float8_e4m3fn)


def _parts(pool, d):
    """Views K codes, V codes, K scales, V scales [pages, heads, 128, .] of a pool."""
    c, s = PAGE * d // 2, PAGE * d // 16
    kc, vc, ks, vs = pool.split([c, c, s, s], -1)
    f8 = torch.float8_e4m3fn
    return (kc.unflatten(-1, (PAGE, d // 2)), vc.unflatten(-1, (PAGE, d // 2)),
            ks.view(f8).unflatten(-1, (PAGE, d // 16)), vs.view(f8).unflatten(-1, (PAGE, d // 16)))


# ---------------------------------------------------------------------------- inputs

def _tables(gen, lens, capacity):
    """A page table [B, capacity] of shuffled pages for the given lengths, and the pool's size."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((len(lens), capacity), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, total


def _positions(case, gen):
    t, far = case["t"], case["far"]
    if case["axes"] == 1:
        if t == far or t > 4096:  # one sequence in order
            return torch.arange(t, device="cuda", dtype=torch.int32)[:, None]
        return torch.randint(0, far, (t, 1), generator=gen, device="cuda").int()
    i = torch.arange(t, device="cuda")  # raster order of a latent with rows of 28 x 56
    return torch.stack((i // (28 * 56), i // 56 % 28, i % 56), 1).int()


def _frequencies(case):
    """(inv_freq fp64, factor of the rotated values, pairs of each axis)."""
    pairs = case["rot"] // 2
    if case["axes"] == 3:
        side = pairs // 3
        count = (pairs - 2 * side, side, side)
        f = [10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in count]
        return torch.cat(f).cuda(), 1.0, count
    f = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    s, mscale = case["factor"], 1.0
    if s > 1:  # scaled by parts: frequencies of under 1 turn in 8192 positions are divided by s
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        f = f / s * (1 - keep) + f * keep
        mscale = 0.1 * math.log(s) + 1
    return f.cuda(), mscale, (pairs,)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st = dict(case)
    if case["op"] == "rope":
        t, hq, hk, d = (case[n] for n in ("t", "hq", "hk", "d"))
        qkv = normal(t, (hq + 2 * hk) * d).to(bf)  # the fused projection's output
        st["q"], st["k"] = qkv[:, :hq * d].view(t, hq, d), qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        st["positions"] = _positions(case, gen)
        st["inv_freq"], st["mscale"], st["pairs"] = _frequencies(case)
    elif case["op"] == "append":
        hkv, d = case["hkv"], case["d"]
        runs = _prompts(case)
        rng.shuffle(runs)
        lens = [n + before for n, before in runs]
        t = sum(n for n, _ in runs)
        kv = normal(t, 2 * hkv * d).to(bf)
        kv[:, ::37] *= 8  # channels of larger values
        st["k"], st["v"] = kv[:, :hkv * d].view(t, hkv, d), kv[:, hkv * d:].view(t, hkv, d)
        st["table"], pages = _tables(gen, lens, (max(lens) + PAGE - 1) // PAGE + 1)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = [0]
        for n, _ in runs:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["pool"] = torch.zeros(pages, hkv, PAGE * d * 9 // 8, dtype=torch.uint8, device="cuda")
    elif case["op"] == "decode":
        b, h, hkv, d = (case[n] for n in ("b", "h", "hkv", "d"))
        lens = _lengths(case)
        rng.shuffle(lens)
        st["table"], pages = _tables(gen, lens, (max(lens) + PAGE - 1) // PAGE + 1)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["pool"] = torch.empty(pages, hkv, PAGE * d * 9 // 8, dtype=torch.uint8, device="cuda")
        for at in range(0, pages, 1024):  # K and V as the append would have left them
            part = st["pool"][at:at + 1024]
            kc, vc, ks, vs = _parts(part, d)
            for codes, scales in ((kc, ks), (vc, vs)):
                c, s = _quantize(normal(*codes.shape[:-1], d).to(bf))
                codes.copy_(_pack(c))
                scales.view(torch.uint8).copy_(s.view(torch.uint8))
        st["q"] = normal(b, h, d).to(bf)
        st["scale"] = d ** -0.5
    else:
        m, n, k = (case[v] for v in "mnk")
        st["x"] = normal(m, k).to(bf)
        w = (normal(n, k) * k ** -0.5).to(bf)
        st["wg"] = 2688.0 / w.abs().amax().float()
        st["xg"] = torch.tensor(2688.0 / 5.5, device="cuda")  # a calibrated input scale
        codes, s8 = _quantize(w, st["wg"])
        st["codes"], st["scales"] = _pack(codes), _tile_scales(s8)
        st["b"] = (normal(n) * 0.1).to(bf) if case["bias"] else None
    return st


# ---------------------------------------------------------------------------- the plain forms

def _plain_rope(st):
    rot, pairs = st["rot"], st["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(len(st["pairs"]), device="cuda"),
                                   torch.tensor(st["pairs"], device="cuda"), output_size=pairs)
    angle = st["positions"].double()[:, axis] * st["inv_freq"]
    c = (angle.cos() * st["mscale"]).float()[:, None]
    s = (angle.sin() * st["mscale"]).float()[:, None]
    if st["inverse"]:
        s = -s

    def turn(x):
        f = x.float()
        if st["interleaved"]:
            a, b = f[..., 0:rot:2], f[..., 1:rot:2]
            y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
        else:
            a, b = f[..., :pairs], f[..., pairs:rot]
            y = torch.cat((a * c - b * s, a * s + b * c), -1)
        return torch.cat((y.to(x.dtype), x[..., rot:]), -1)

    return turn(st["q"]), turn(st["k"])


def _plain_append(st):
    d, t = st["d"], st["k"].shape[0]
    row = torch.arange(t, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(st["cu"], row, right=True) - 1
    pos = st["lens"][seq] - st["cu"][seq + 1] + row
    pos = torch.where(pos >= 0, pos, torch.zeros_like(pos) - 1)
    live = pos >= 0
    page = st["table"][seq, pos.clamp(min=0) // PAGE]
    page, slot = page[live].long(), (pos % PAGE)[live].long()
    kc, vc, ks, vs = _parts(st["pool"], d)
    for x, codes, scales in ((st["k"], kc, ks), (st["v"], vc, vs)):
        c, s = _quantize(x[live])
        codes[page, :, slot] = _pack(c)
        scales.view(torch.uint8)[page, :, slot] = s.view(torch.uint8)


def _mask(st, n):
    pos = torch.arange(n, device="cuda")
    lens = st["lens"][:, None]
    seen = pos < lens
    if st["window"]:
        seen = seen & ((pos >= lens - st["window"]) | (pos < st["sinks"]))
    return seen


def _plain_decode(st):
    b, h, hkv, d = (st[n] for n in ("b", "h", "hkv", "d"))
    pages = st["pool"][st["table"].clamp(min=0).long()]  # [B, P, Hkv, record]
    n = pages.shape[1] * PAGE
    kc, vc, ks, vs = (p.transpose(1, 2).flatten(2, 3) for p in _parts(pages, d))  # [B, Hkv, n, .]
    qc, qs = _quantize(st["q"])
    q = _unpack(_pack(qc), qs).view(b, hkv, h // hkv, d)
    s = (q @ _unpack(kc, ks).mT) * st["scale"]
    seen = _mask(st, n)[:, None, None]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    l = p.sum(-1, keepdim=True)
    acc = p @ _unpack(vc, vs)
    o = torch.where(l > 0, acc / l, torch.zeros_like(acc))
    return o.view(b, h, d).to(torch.bfloat16), (m + l.log()).view(b, h)


def _plain_linear(st):
    n, k = st["n"], st["k"]
    w = _unpack(st["codes"], _untile_scales(st["scales"], n, k // 16))
    c, s = _quantize(st["x"], st["xg"])
    out = (_unpack(_pack(c), s) @ w.T) * (1.0 / (st["wg"] * st["xg"]))
    return (out if st["b"] is None else out + st["b"].float()).to(torch.bfloat16)


# ---------------------------------------------------------------------------- one pass

def _cache(st):
    """The pool as what it holds: code bytes and scale values."""
    kc, vc, ks, vs = _parts(st["pool"], st["d"])
    return dict(k_codes=kc, v_codes=vc, k_scales=ks, v_scales=vs)


def run(state):
    st, op = state, state["op"]
    if own:
        from nvfp4_fake_quant_gb300 import api
        if op == "rope":
            return api.rope_apply(st["q"], st["k"], st["positions"], st["inv_freq"],
                                  interleaved=st["interleaved"], axis_pairs=st["pairs"],
                                  mscale=st["mscale"], inverse=st["inverse"])
        if op == "append":
            api.nvfp4_kv_append(st["k"], st["v"], st["lens"], st["table"], st["pool"],
                                cu_tokens=st["cu"] if st["prompt"] else None)
            return _cache(st)
        if op == "decode":
            if "ws" not in st:  # kept by a serving loop, as the pool is
                st["ws"] = torch.empty(api.attn_qat_decode_workspace(
                    st["b"], st["h"], st["hkv"], st["d"], st["table"].shape[1]),
                    dtype=torch.uint8, device="cuda")
            return api.attn_qat_decode(st["q"], st["pool"], st["table"], st["lens"],
                                       scale=st["scale"], window=st["window"], sinks=st["sinks"],
                                       workspace=st["ws"])
        if "ws" not in st:
            st["ws"] = torch.empty(api.nvfp4_linear_packed_workspace(st["m"], st["n"], st["k"]),
                                   dtype=torch.uint8, device="cuda")
        return api.nvfp4_linear_packed_fwd(st["x"], st["codes"], st["scales"], st["wg"],
                                           bias=st["b"], x_global_sf=st["xg"], workspace=st["ws"])
    if op == "rope":
        return _plain_rope(st)
    if op == "append":
        _plain_append(st)
        return _cache(st)
    return _plain_decode(st) if op == "decode" else _plain_linear(st)


# ---------------------------------------------------------------------------- in 64 bits

def _codes64(x, g):
    """(values before the division by g, scales), fp64, of the NVFP4 decisions on x: the scale's
    and the elements' roundings by distance to the nearest representable value, ties to the even."""
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
    if g is not None:
        blk = blk * g  # the definition decides on this fp32 product and the fp32 quotients
    top = blk.abs().max(-1).values
    s = nearest((top / torch.tensor([6.0], device=x.device)).double(), e4m3)
    q = (blk.abs() / s.float()[..., None]).nan_to_num(0.0, posinf=0.0).double()
    return (torch.copysign(nearest(q, e2m1), blk.double()) * s[..., None]).reshape(x.shape), s


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


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        rot, inter = st["rot"], st["interleaved"]
        first = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
        second = first + (1 if inter else rot // 2)
        cols, at = [], 0
        for axis, n in enumerate(st["pairs"]):
            cols.append(st["positions"][:, axis:axis + 1].double() * st["inv_freq"][at:at + n])
            at += n
        z = torch.polar(torch.full((), float(st["mscale"]), dtype=torch.float64, device="cuda"),
                        torch.cat(cols, 1))[:, None]
        z = z.conj() if st["inverse"] else z
        out = []
        for x in (st["q"], st["k"]):
            y = x.double()
            w = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = w.real, w.imag
            out.append(y)
        return tuple(out)
    if case["op"] == "append":
        got = {}
        for name, x in (("k", st["k"]), ("v", st["v"])):
            s = _codes64(x, None)[1]
            out = torch.zeros(st["pool"].shape[0], st["hkv"], PAGE, st["d"] // 16,
                              dtype=torch.float64, device="cuda")
            for i, n in enumerate(st["lens"].tolist()):
                a, e = st["cu"][i:i + 2].tolist()
                if n:
                    pos = torch.arange(n - (e - a), n, device="cuda")
                    out[st["table"][i, pos // PAGE].long(), :, pos % PAGE] = s[a:e]
            got[name + "_codes"], got[name + "_scales"] = None, out
        return got
    if case["op"] == "linear":
        n, k = st["n"], st["k"]
        sw = torch.empty(n, k // 16, dtype=torch.uint8, device="cuda")
        r, c = torch.arange(n, device="cuda")[:, None], torch.arange(k // 16, device="cuda")
        at = ((r // 128) * ((k // 16 + 3) // 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4
        sw = st["scales"][at]
        y = _codes64(st["x"], st["xg"])[0] @ _bytes64(st["codes"], sw).T
        y = y / (st["wg"].double() * st["xg"].double())
        return y if st["b"] is None else y + st["b"].double()
    h, hkv, d = case["h"], case["hkv"], case["d"]
    q = _codes64(st["q"], None)[0].view(-1, hkv, h // hkv, d)
    o = torch.zeros(case["b"], h, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["b"], h), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(st["lens"].tolist()):
        if n:
            rec = st["pool"][st["table"][i, :(n + PAGE - 1) // PAGE].long()]
            keep = [p for p in range(n) if not case["window"] or p >= n - case["window"] or
                    p < case["sinks"]]
            keep = torch.tensor(keep, device="cuda")
            kc, vc, ks, vs = (x.transpose(0, 1).reshape(hkv, -1, x.shape[-1])[:, keep]
                              for x in _parts(rec, d))
            s = torch.einsum("hgd,hnd->hgn", q[i], _bytes64(kc, ks)) * st["scale"]
            o[i] = torch.einsum("hgn,hnd->hgd", s.softmax(-1), _bytes64(vc, vs)).view(h, d)
            lse[i] = s.logsumexp(-1).view(h)
    return o, lse
