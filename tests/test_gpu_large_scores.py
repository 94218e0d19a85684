"""Scores so large that fp32 has no digits left for their differences: p, rounded to f16, must not
become infinite (it would be NaN in the output).

The keys of a sequence agree in all elements but 16, so scores of up to 2^30 differ by a few units
or by their rounding.  Nothing is said about which key wins there: every output is a mean of V,
inside V's range up to its rounding to bf16 and p's to f16 (2^-8 + 2^-11 + 2^-12 of the largest
|V|), and lse is a score of some key up to the rounding, 2^-16 of it, and ln of the keys' number.
"""
import math

import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_cross import ints, offsets
from test_gpu_kv_cache import BF16, PAGE

pytestmark = pytest.mark.gpu
PAGES = 12


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [2.0 ** -4, 1.0, 37.0])
@pytest.mark.parametrize("size", [30.0, 300.0, 2688.0])
def test_outputs_are_means(d, scale, size):
    h, hkv, n = 6, 3, PAGES * PAGE - 3
    g = torch.Generator().manual_seed(d + int(size))
    sign = torch.randn(d, generator=g).sign()
    k = (sign * size).expand(PAGES, hkv, PAGE, d).clone()
    k[..., -16:] = torch.randn(PAGES, hkv, PAGE, 16, generator=g) * size / 64
    v = torch.randn(PAGES, hkv, PAGE, d, generator=g)
    pool = torch.empty(PAGES, hkv, 144 * d, dtype=torch.uint8)
    for x, at_c, at_s in ((k, 0, 128 * d), (v, 64 * d, 136 * d)):
        c, s = os_.pack(x.to(BF16))
        pool[:, :, at_c:at_c + 64 * d], pool[:, :, at_s:at_s + 8 * d] = c.flatten(2), s.flatten(2)
    kc, vc, ks, vs = os_.record_parts(pool, d)
    keys = os_.unpack(kc, ks).transpose(0, 1).flatten(1, 2)[:, :n]
    vals = os_.unpack(vc, vs).transpose(0, 1).flatten(1, 2)[:, :n]
    lo, hi = (f(vals, 1).repeat_interleave(2, 0) for f in (torch.amin, torch.amax))  # [H, D]
    slack = float(vals.abs().max()) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12)

    def check(o, lse, q, several):
        o, lse = o.cpu().double(), lse.cpu().double()
        s = torch.stack([os_.fq(q[:, x]) @ keys[x // 2].T for x in range(h)], 1) * scale
        assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
        assert bool(((o >= lo - slack) & (o <= hi + slack)).all())
        off = s.abs().amax(-1) * 2.0 ** -16 + 2.0 ** -20
        assert bool((lse >= s.amax(-1) - off).all())
        assert bool((lse <= s.amax(-1) + math.log(several) + off).all())

    table, pool = torch.arange(PAGES).int()[None].cuda(), pool.cuda()
    for t in (3, 300):
        q = (sign * size * (1 + torch.rand(t, h, 1, generator=g) / 8)).to(BF16)
        q[..., -16:] = torch.randn(t, h, 16, generator=g).to(BF16)
        o, lse = api.attn_qat_cross(q.cuda(), pool, table, ints([n]), ints(offsets([t])), scale)
        check(o, lse, q, n)
        q = q[:40]
        b = len(q)
        o, lse = api.attn_qat_decode(q.cuda(), pool, table.expand(b, -1).contiguous(), ints([n] * b),
                                     scale)
        check(o, lse, q, n)
        o, lse = api.attn_qat_decode_prefix(q.cuda(), pool, table[:, 3:5].expand(b, -1).contiguous(),
                                            ints([200] * b), table, ints([n]), scale=scale)
        check(o, lse, q, n + 200)
    assert api.device_status() == 0
