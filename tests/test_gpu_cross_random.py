"""Random ragged shapes: attention of many rows, and of single tokens behind prefixes, against
attn_qat_decode on a sequence for each row; every call twice for equal bits, on workspaces and
into outputs of NaN.  Row counts of one and two halves of a tile follow each other, some sequences
have no rows or no keys, pages are shared.

Bounds: both sides keep those of test_gpu_kv_cache.py, |o| 2^-8 + A (2^-11 + 2^-12) +
n 2^-32 vmax + 2 A E 2^-16 with A <= vmax, and E 2^-16 + 2^-20 + |lse| 2^-23 for lse, so their
difference twice that.  E: scale max_j sum |q~ k~_j| over all keys of the pool.
"""
import random

import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_cross import ints, offsets, vmax_of
from test_gpu_kv_cache import BF16, PAGE, check_decode, make_pool

pytestmark = pytest.mark.gpu
PAGES, WIDE = 16, 12
SHAPES = 40


def close(got, want, e, n, vmax):
    (o, lse), (o2, lse2) = got, want
    es = e * 2.0 ** -16
    o, o2, fin = o.double(), o2.double(), torch.isfinite(lse2)
    tol = 2 * (o2.abs() * 2.0 ** -8 + vmax * (2.0 ** -11 + 2.0 ** -12 + n * 2.0 ** -32) +
               2 * vmax * es[..., None])
    # of the reference's bf16 value in place of the exact one: half a step of it more
    assert bool(((o - o2).abs() <= tol * (1 + 2.0 ** -7)).all())
    assert torch.equal(torch.isfinite(lse), fin) and not bool(o[~fin].any())
    d = (lse - lse2).abs().double()[fin]
    assert bool((d <= (2 * (es + 2.0 ** -20 + lse2.abs() * 2.0 ** -23))[fin]).all())


def twice(call, ws_bytes, t, h, d):
    got = []
    for _ in range(2):
        ws = torch.full((ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        o = torch.full((t, h, d), float("nan"), dtype=BF16, device="cuda")
        lse = torch.full((t, h), float("nan"), device="cuda")
        got.append(call(o=o, lse=lse, workspace=ws))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    return got[0]


@pytest.mark.parametrize("seed,d,hkv", [(s, d, hkv) for s, (d, hkv) in enumerate(
    (d, hkv) for d in (64, 128) for hkv in (1, 2, 3, 8))])
def test_random_shapes(seed, d, hkv):
    rng = random.Random(seed)
    gen = torch.Generator().manual_seed(seed)
    pool = make_pool(PAGES, hkv, d, gen)
    vmax = vmax_of(pool, d)
    kc, _, ks, _ = os_.record_parts(pool, d)
    keys = os_.unpack(kc, ks).abs().transpose(0, 1).flatten(1, 2).float().cuda()  # [Hkv, keys, D]
    pool, scale = pool.cuda(), d ** -0.5
    for _ in range(SHAPES):
        g = rng.choice((1, 1, 2, 4, 5, 8, 16, 32))
        b, h = rng.choice((1, 2, 3, 5, 9, 40, 200)), hkv * g
        most = max(2, min(900, 6000 // (b * h)))
        toks = [rng.choice((0, 1, rng.randint(0, most), rng.randint(0, max(1, 300 // g))))
                for _ in range(b)]
        if sum(toks) == 0:
            toks[-1] = 1
        lens = [rng.choice((0, 1, PAGE, rng.randint(0, 300), rng.randint(0, WIDE * PAGE)))
                for _ in range(b)]
        t = sum(toks) + rng.choice((0, 0, 3))
        table = torch.randint(0, PAGES, (b, WIDE), generator=gen).int().cuda()
        q = (torch.randn(t, h, d, generator=gen) * rng.choice((0.3, 1, 3))).to(BF16)
        seq = torch.repeat_interleave(torch.arange(b), torch.tensor(toks)).cuda()
        m, n = len(seq), ints(lens)
        e = torch.stack([(os_.fq(q[:m, x]).abs().float().cuda() @ keys[x // g].T).amax(-1)
                         for x in range(h)], 1).double() * scale
        q = q.cuda()
        o, lse = twice(lambda **k: api.attn_qat_cross(q, pool, table, n, ints(offsets(toks)), **k),
                       api.attn_qat_cross_workspace(t, b, h, hkv, d, WIDE), t, h, d)
        want = api.attn_qat_decode(q[:m], pool, table[seq], n[seq])
        close((o[:m], lse[:m]), want, e, WIDE * PAGE, vmax)
        assert not bool(o[m:].any()) and bool((lse[m:] == -float("inf")).all())
        # the first rows as single tokens behind their sequences' whole pages as prefixes
        r = min(m, 200)
        own = torch.randint(0, 400, (r,), generator=gen).int().cuda()
        own[::7] = 0
        mine, shared = torch.randint(0, PAGES, (r, 4), generator=gen).int().cuda(), n // PAGE * PAGE
        groups = torch.searchsorted(seq[:r].contiguous(), torch.arange(b + 1, device="cuda")).int()
        o, lse = twice(lambda **k: api.attn_qat_decode_prefix(q[:r], pool, mine, own, table, shared,
                                                              groups, **k),
                       api.attn_qat_decode_prefix_workspace(r, b, h, hkv, d, 4, WIDE), r, h, d)
        page, first = torch.arange(WIDE + 4, device="cuda")[None], (shared // PAGE)[seq[:r]][:, None]
        both = torch.where(page < first, table[seq[:r]].gather(1, page.expand(r, -1).clamp(max=WIDE - 1)),
                           mine.gather(1, (page - first).clamp(0, 3)))
        want = api.attn_qat_decode(q[:r], pool, both.int(), own + shared[seq[:r]])
        close((o, lse), want, e[:r], (WIDE + 4) * PAGE, vmax)
        assert api.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 100, 128])
def test_one_run(d, n):
    """A table of one page and one KV head: a grid of one run."""
    gen = torch.Generator().manual_seed(n)
    pool, table, q = make_pool(2, 1, d, gen), ints([[1]]), torch.randn(5, 3, d, generator=gen).to(BF16)
    ref = os_.attend(q, pool, [(table[0], n)], d ** -0.5)
    for more in ((), (ints([0, 5]),)):
        o, lse = api.attn_qat_cross(q.cuda(), pool.cuda(), table, ints([n]), *more)
        check_decode(o, lse, ref, n, vmax_of(pool, d))
    assert api.device_status() == 0
