"""Offsets that decrease: sequences would have rows in common, so none has any; offsets outside of
the rows only are cut.  Every output is defined, and the same in every call."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from test_gpu_cross import ints, offsets, queries, reference, vmax_of
from test_gpu_kv_cache import BF16, check_decode, make_pool, tables

pytestmark = pytest.mark.gpu


def twice(call, t, h, d):
    """The outputs of a call, which two calls into buffers of NaN have to agree on; status 1."""
    got = []
    for _ in range(2):
        o = torch.full((t, h, d), float("nan"), dtype=BF16, device="cuda")
        lse = torch.full((t, h), float("nan"), device="cuda")
        call(o=o, lse=lse)
        assert api.device_status() == 1 and api.device_status() == 0
        got.append((o, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    return got[0]


@pytest.mark.parametrize("h,hkv,d", [(4, 2, 64), (12, 12, 128)])
@pytest.mark.parametrize("cu", [[0, 700, 30, 900], [900, 0, 900, 900], [0, 900, 900, 0],
                                [-3, 1000, 899, 2000], [0, 300, 299, 299]], ids=str)
def test_cross(h, hkv, d, cu):
    g = torch.Generator().manual_seed(h)
    lens, t = [300, 0, 500], 900
    table, pages = tables(lens, 4, g)
    args = (queries(t, h, d, g).cuda(), make_pool(pages, hkv, d, g).cuda(), table.clamp(0, 0).cuda(),
            ints(lens), ints(cu))
    o, lse = twice(lambda **k: api.attn_qat_cross(*args, **k), t, h, d)
    assert not bool(o.any()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("b,at", [(641, 640), (641, 641), (641, 639), (1500, 700), (1500, 701), (2000, 1)])
def test_cross_of_many_sequences(b, at):
    """The one offset that decreases anywhere in the list, the others as they should be.  (641, 640)
    is an offset outside of the rows: cut to the rows' end it is the next one, and no decrease."""
    h, hkv, d = 2, 1, 64
    g = torch.Generator().manual_seed(b)
    pool, table = make_pool(4, hkv, d, g).cuda(), torch.randint(0, 4, (b, 2), generator=g).int().cuda()
    cu = offsets([1] * b)
    q = queries(b, h, d, g).cuda()
    lens = ints([130] * b)
    ok = api.attn_qat_cross(q, pool, table, lens, ints(cu))
    assert bool(torch.isfinite(ok[1]).all()) and api.device_status() == 0
    cu[at] = cu[at + 1] + 1 if at < b else cu[at - 1] - 1
    o, lse = twice(lambda **k: api.attn_qat_cross(q, pool, table, lens, ints(cu), **k), b, h, d)
    if all(min(x, b) <= min(y, b) for x, y in zip(cu, cu[1:])):
        assert (b, at) == (641, 640)
        cut = [min(x, b) for x in cu]
        ref = reference(q.cpu(), pool.cpu(), table.cpu(), [130] * b, cut, d ** -0.5)
        return check_decode(o, lse, ref, 130, vmax_of(pool.cpu(), d))
    assert not bool(o.any()) and bool((lse == -float("inf")).all())


def test_cross_with_offsets_outside_of_the_rows():
    h, hkv, d, t = 4, 2, 64, 90
    g = torch.Generator().manual_seed(3)
    lens = [200, 130, 7]
    table, pages = tables(lens, 2, g)
    pool, q = make_pool(pages, hkv, d, g), queries(t, h, d, g)
    for cu in ([-5, 20, 70, 80], [3, 20, 20, 1 << 30], [-(1 << 31), -7, 95, (1 << 31) - 1]):
        ref = reference(q, pool, table, lens, [min(max(x, 0), t) for x in cu], 0.125)
        args = (q.cuda(), pool.cuda(), table.cuda(), ints(lens), ints(cu), 0.125)
        o, lse = twice(lambda **k: api.attn_qat_cross(*args, **k), t, h, d)
        check_decode(o, lse, ref, max(lens), vmax_of(pool, d))


@pytest.mark.parametrize("cu", [[0, 5, 2, 7], [7, 0, 0, 0], [0, 9, 6, 6]], ids=str)
def test_groups_behind_prefixes(cu):
    """No sequence has a prefix: the decode over its own keys, bit for bit."""
    h, hkv, d, b = 8, 2, 128, 7
    g = torch.Generator().manual_seed(7)
    pool = make_pool(20, hkv, d, g).cuda()
    mine = torch.randint(0, 20, (b, 3), generator=g).int().cuda()
    own, shared = ints([0, 5, 384, 130, 1, 0, 200]), ints([900, 128, 300])
    prefix = torch.randint(0, 20, (3, 8), generator=g).int().cuda()
    q = queries(b, h, d, g).cuda()
    want = api.attn_qat_decode(q, pool, mine, own)
    got = twice(lambda **k: api.attn_qat_decode_prefix(q, pool, mine, own, prefix, shared, ints(cu),
                                                       **k), b, h, d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
