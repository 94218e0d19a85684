"""Keys far below a row's best one, where they are all that the output consists of.

The first key (an attention sink) scores 19 to 27 (log2) above all others and has V = 0; the
others have V > 0.  p = 2^(S - S_max) of the others is 2^-19 to 2^-27, below f16's normal range and
in part below its smallest number, while their sum over a few thousand keys is the whole output.

Bounds per element as in test_gpu_kv_cache.py, with p times 2^7 when it is rounded to f16 (at most
2^15, as scores may exceed the reference maximum by 2^8): half a step of numbers below the normal
range is 2^-25 of p 2^7, hence 2^-32 of p, for each of n keys.
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_cross import ints, vmax_of
from test_gpu_kv_cache import BF16, PAGE

pytestmark = pytest.mark.gpu
PAGES = 24


def sink_pool(hkv, d, g, spread=1.0):
    """PAGES pages: key 0 of page 0 scores about 16 (nats) above the rest for rows of ones and
    scale d^-0.5; its V is 0, the others' V are above 0, of mean 1 where their spread is less."""
    pool = torch.empty(PAGES, hkv, 144 * d, dtype=torch.uint8)
    k = torch.randn(PAGES, hkv, PAGE, d, generator=g) * 0.2
    v = torch.randn(PAGES, hkv, PAGE, d, generator=g).abs() * spread + max(0.1, 1 - spread)
    k[0, :, 0], v[0, :, 0] = 16.2 * d ** -0.5, 0.0
    for x, at_c, at_s in ((k, 0, 128 * d), (v, 64 * d, 136 * d)):
        c, s = os_.pack(x.to(BF16))
        pool[:, :, at_c:at_c + 64 * d], pool[:, :, at_s:at_s + 8 * d] = c.flatten(2), s.flatten(2)
    return pool


def rows(t, h, d):
    """Rows of 0.88 to 1.1 (quantized, 0.84 to 1.12): the gap in the scores goes from 19 to 27 (log2)."""
    return torch.linspace(0.88, 1.1, t * h).view(t, h, 1).expand(t, h, d).to(BF16).contiguous()


def check(o, lse, ref, n, vmax):
    r, l, mag, e = ref
    es = e[..., None] * 2.0 ** -16
    tol = r.abs() * 2.0 ** -8 + mag * (2.0 ** -11 + 2.0 ** -12) + n * 2.0 ** -32 * vmax + 2 * mag * es
    err = (o.cpu().double() - r).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    el = (lse.cpu().double() - l).abs()
    assert bool((el <= es[..., 0] + 2.0 ** -20 + l.abs() * 2.0 ** -23).all()), float(el.max())


def test_the_inputs_are_what_they_should_be():
    g = torch.Generator().manual_seed(1)
    pool, q = sink_pool(2, 64, g), rows(200, 2, 64)
    kc, _, ks, _ = os_.record_parts(pool, 64)
    k = os_.unpack(kc, ks).transpose(0, 1).flatten(1, 2)  # [2, keys, 64]
    s = torch.einsum("thd,hnd->thn", os_.fq(q), k) * 0.125 / torch.log(torch.tensor(2.0))
    gap = s[..., :1] - s[..., 1:]
    assert bool((s.argmax(-1) == 0).all()) and 18 < float(gap.min())
    assert float(gap.mean(-1).min()) < 21 and 25 < float(gap.mean(-1).max()) < 28


@pytest.mark.parametrize("t,h,hkv,d", [(100, 64, 64, 128), (100, 64, 64, 64), (700, 24, 24, 128),
                                       (300, 24, 24, 64), (40, 96, 24, 128)])
def test_cross(t, h, hkv, d):
    g = torch.Generator().manual_seed(t + d)
    pool, q = sink_pool(hkv, d, g), rows(t, h, d)
    table, n = torch.arange(PAGES, dtype=torch.int32)[None], PAGES * PAGE - 5
    ref = os_.attend(q, pool, [(table[0], n)], d ** -0.5)
    o, lse = api.attn_qat_cross(q.cuda(), pool.cuda(), table.cuda(), ints([n]))
    check(o, lse, ref, n, vmax_of(pool, d))
    assert api.device_status() == 0


@pytest.mark.parametrize("h,hkv,d", [(64, 64, 64), (64, 16, 128)])
@pytest.mark.parametrize("own", [0, 200])
def test_behind_a_prefix_that_begins_with_it(h, hkv, d, own):
    g = torch.Generator().manual_seed(h + d)
    b = 30
    pool, q = sink_pool(hkv, d, g), rows(b, h, d)
    prefix, n = torch.arange(PAGES, dtype=torch.int32)[None], PAGES * PAGE
    mine = torch.tensor([[5, 9]], dtype=torch.int32)
    ref = os_.attend(q, pool, [(prefix[0], n), (mine[0], own)], d ** -0.5)
    o, lse = api.attn_qat_decode_prefix(q.cuda(), pool.cuda(), mine.expand(b, 2).contiguous().cuda(),
                                        ints([own] * b), prefix.cuda(), ints([n]))
    check(o, lse, ref, n + own, vmax_of(pool, d))
    assert api.device_status() == 0


@pytest.mark.parametrize("h,hkv,d", [(8, 8, 64), (16, 8, 128), (36, 3, 64)])
def test_single_tokens(h, hkv, d):
    """40 sequences of the same keys: runs hold most of a segment."""
    g = torch.Generator().manual_seed(h + d)
    b, n = 40, PAGES * PAGE - 5
    pool, q = sink_pool(hkv, d, g, spread=0.1), rows(b, h, d)
    table = torch.arange(PAGES, dtype=torch.int32)[None]
    ref = os_.attend(q, pool, [(table[0], n)], d ** -0.5)
    args = (q.cuda(), pool.cuda(), table.expand(b, -1).contiguous().cuda(), ints([n] * b))
    for call in (api.attn_qat_decode, api.attn_qat_cross):
        o, lse = call(*args)
        check(o, lse, ref, n, vmax_of(pool, d))
    # the same as own keys behind a prefix of some of the others
    prefix = torch.tensor([[3, 7, 8]], dtype=torch.int32)
    ref = os_.attend(q, pool, [(prefix[0], 300), (table[0], n)], d ** -0.5)
    o, lse = api.attn_qat_decode_prefix(*args, prefix.cuda(), ints([300]))
    check(o, lse, ref, n + 300, vmax_of(pool, d))
    assert api.device_status() == 0
