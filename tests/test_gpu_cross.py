"""Attention of many rows over the paged cache (attn_qat_cross) and single tokens behind a
shared prefix (attn_qat_decode_prefix) against oracle/serving.py.

Bounds per element, those of test_gpu_kv_cache.py: half a bf16 step of the result, p rounded to
f16 with fp32 exponentials and sums, p below f16's normal range, the fp32 sums of S.  The sums of
p V~ add 16 products at a time into fp32: n / 16 steps of 2^-23 at most of sum p |v| / l, below
2^-12 up to 32768 keys and inside the bound's share for fp32 sums.  Two parts that meet add an
fp32 rounding of each logarithm (2^-24 |lse|, in the bound of lse) and of the products.
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_kv_cache import BF16, PAGE, check_decode, make_pool, spoil, tables

pytestmark = pytest.mark.gpu


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(counts, first=0):
    got = [first]
    for n in counts:
        got.append(got[-1] + n)
    return got


def vmax_of(pool, d):
    return float(os_.unpack(*os_.record_parts(pool, d)[1::2]).abs().max())


def queries(t, h, d, g, pad=16):
    """bf16 [t, h, d] with strided rows."""
    return torch.randn(t, h * d + pad, generator=g).to(BF16)[:, :h * d].unflatten(1, (h, d))


def reference(q, pool, table, lens, cu, scale):
    """attend for every sequence's rows; rows outside all of them as rows without keys."""
    t, h, d = q.shape
    out = (torch.zeros(t, h, d, dtype=torch.float64),
           torch.full((t, h), -float("inf"), dtype=torch.float64),
           torch.zeros(t, h, d, dtype=torch.float64), torch.zeros(t, h, dtype=torch.float64))
    for i, n in enumerate(lens):
        r = slice(cu[i], cu[i + 1])
        for x, y in zip(out, os_.attend(q[r], pool, [(table[i], n)], scale)):
            x[r] = y
    return out


CASES = [  # h, hkv, d, tokens, lengths
    (1, 1, 128, [1], [1]), (1, 1, 64, [2], [129]), (4, 4, 64, [5, 1, 3, 2], [128, 1, 127, 300]),
    (8, 2, 128, [31, 0, 33, 64], [300, 5, 0, 641]), (7, 1, 128, [37, 2], [1000, 0]),
    (12, 12, 128, [130], [512]), (16, 1, 64, [17, 8, 9], [700, 17, 256]),
    (24, 2, 64, [11, 11], [383, 385]), (40, 1, 128, [7], [130]), (2, 1, 128, [700], [64]),
    (3, 3, 64, [129, 255, 1], [128, 256, 2000]), (1, 1, 128, [9], [5000]), (1, 1, 64, [400], [4100]),
    (32, 1, 128, [9, 40], [300, 100]), (64, 2, 64, [3, 70], [130, 128]), (8, 8, 128, [100, 33], [128, 1]),
    (96, 2, 64, [5, 11], [100, 260]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}_{c[3][0]}_{c[4][0]}")
def test_cross_parity(case):
    h, hkv, d, toks, lens = case
    g = torch.Generator().manual_seed(sum(lens) + h)
    table, pages = tables(lens, -(-max(lens) // PAGE) + 2, g)
    pool = make_pool(pages, hkv, d, g)
    vmax = vmax_of(pool, d)
    spoil(pool, table, lens, d)
    first, t = 3, sum(toks) + 8  # rows before the first and behind the last sequence
    cu = offsets(toks, first)
    q = queries(t, h, d, g)
    ref = reference(q, pool, table, lens, cu, d ** -0.5)
    # a workspace of arbitrary bytes (NaN patterns), the second call on the first's
    ws = torch.full((api.attn_qat_cross_workspace(t, len(lens), h, hkv, d, table.shape[1]),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    args = (q.cuda(), pool.cuda(), table.cuda(), ints(lens), ints(cu))
    o = torch.full((t, h, d), float("nan"), dtype=BF16, device="cuda")
    lse = torch.full((t, h), float("nan"), device="cuda")
    api.attn_qat_cross(*args, o=o, lse=lse, workspace=ws)
    assert api.device_status() == 0
    check_decode(o, lse, ref, max(lens), vmax)
    o2, lse2 = api.attn_qat_cross(*args, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("h,hkv,d,n,lens", [
    (4, 2, 64, 1, [300, 0, 128, 5]), (4, 2, 128, 2, [300, 0, 128]), (6, 6, 64, 130, [77, 140])])
def test_equal_groups_without_offsets(h, hkv, d, n, lens):
    """The call without offsets is the call with them (one token a sequence: another kernel)."""
    g = torch.Generator().manual_seed(n)
    table, pages = tables(lens, 4, g)
    pool = make_pool(pages, hkv, d, g)
    q = queries(n * len(lens), h, d, g)
    cu = offsets([n] * len(lens))
    args = (q.cuda(), pool.cuda(), table.cuda(), ints(lens))
    ref = reference(q, pool, table, lens, cu, d ** -0.5)
    for more in ((), (ints(cu),)):
        o, lse = api.attn_qat_cross(*args, *more)
        check_decode(o, lse, ref, max(lens), vmax_of(pool, d))
    assert api.device_status() == 0


@pytest.mark.parametrize("h,hkv,d,b,most,longest", [
    (2, 1, 64, 700, 3, 300), (8, 2, 128, 90, 40, 600), (4, 4, 64, 40, 200, 900),
    (3, 1, 128, 1100, 2, 200)])
def test_cross_of_many_sequences(h, hkv, d, b, most, longest):
    """More segments than the chip has runs, pages shared, the table a slice of a wider one."""
    g = torch.Generator().manual_seed(b + h)
    lens = torch.randint(0, longest + 1, (b,), generator=g).tolist()
    toks = torch.randint(0, most + 1, (b,), generator=g).tolist()
    lens[b // 2], toks[b // 2] = longest, most
    width = -(-longest // PAGE)
    pool = make_pool(40, hkv, d, g)
    wide = torch.randint(0, 40, (b, width + 3), generator=g, dtype=torch.int32)
    cu = offsets(toks)
    q = queries(cu[-1], h, d, g)
    ref = reference(q, pool, wide, lens, cu, d ** -0.5)
    args = (q.cuda(), pool.cuda(), wide.cuda()[:, :width], ints(lens), ints(cu))
    o, lse = api.attn_qat_cross(*args)
    check_decode(o, lse, ref, longest, vmax_of(pool, d))
    o2, lse2 = api.attn_qat_cross(*args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and api.device_status() == 0


def rising_pool(pages, d, g):
    """Keys that grow along the pages in one direction: with the query in it, scores rise from
    page to page (the reference maximum is raised again and again)."""
    k = torch.randn(pages, 1, PAGE, d, generator=g) * 0.1
    k += torch.arange(pages)[:, None, None, None] / 2
    pool = make_pool(pages, 1, d, g)
    c, s = os_.pack(k.to(BF16))
    pool[:, :, :64 * d], pool[:, :, 128 * d:136 * d] = c.flatten(2), s.flatten(2)
    return pool


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rising_and_falling_scores(d, sign):
    g = torch.Generator().manual_seed(d)
    pool = rising_pool(20, d, g)
    q = (torch.randn(300, 1, d, generator=g) * 0.2 + sign).to(BF16)
    table, lens = torch.arange(20, dtype=torch.int32)[None], [20 * PAGE - 5]
    ref = reference(q, pool, table, lens, [0, 300], 0.5)
    o, lse = api.attn_qat_cross(q.cuda(), pool.cuda(), table.cuda(), ints(lens), scale=0.5)
    check_decode(o, lse, ref, lens[0], vmax_of(pool, d))
    # the same keys behind each other as a prefix and own tokens, in both orders
    for lo, hi in ((12, 8), (1, 19)):
        for first, second in ((range(lo), range(lo, 20)), (range(lo, 20), range(lo))):
            a, b = (torch.tensor([list(x)], dtype=torch.int32) for x in (first, second))
            r = os_.attend(q[:3], pool, [(a[0], a.numel() * PAGE), (b[0], b.numel() * PAGE)], 0.5)
            o, lse = api.attn_qat_decode_prefix(
                q[:3].cuda(), pool.cuda(), b.expand(3, -1).contiguous().cuda(),
                ints([b.numel() * PAGE] * 3), a.cuda(), ints([a.numel() * PAGE]), scale=0.5)
            check_decode(o, lse, r, 20 * PAGE, vmax_of(pool, d))
    assert api.device_status() == 0


def test_sharp_and_flat_scores():
    d, n = 64, 1500
    g = torch.Generator().manual_seed(3)
    table, pages = tables([n], 12, g)
    pool = make_pool(pages, 1, d, g)
    q = torch.randn(140, 2, d, generator=g).to(BF16)
    for scale in (30.0, 1e-3):
        ref = reference(q, pool, table, [n], [0, 140], scale)
        o, lse = api.attn_qat_cross(q.cuda(), pool.cuda(), table.cuda(), ints([n]), scale=scale)
        check_decode(o, lse, ref, n, vmax_of(pool, d))
    assert api.device_status() == 0


def test_bad_pages_lengths_and_offsets_are_left_out_and_reported():
    d, lens = 64, [300, 200, 130]
    g = torch.Generator().manual_seed(4)
    table, pages = tables(lens, 3, g)
    pool = make_pool(pages, 2, d, g)
    vmax = vmax_of(pool, d)
    table[0, 0], table[1, 1], table[2, 0], table[2, 1] = -1, pages, 1 << 30, -7
    cu = [0, 70, 71, 90]
    q = torch.randn(90, 4, d, generator=g).to(BF16)
    gone = {(0, 0), (1, 1), (2, 0), (2, 1)}
    ref = tuple(torch.cat(x) for x in zip(*(
        os_.attend(q[cu[i]:cu[i + 1]], pool, [(table[i].clamp(0, pages - 1), lens[i])], 0.125,
                   keep=lambda _, j, i=i: (i, j // PAGE) not in gone) for i in range(3))))
    args = (q.cuda(), pool.cuda(), table.cuda(), ints(lens))
    o, lse = api.attn_qat_cross(*args, ints(cu), 0.125)
    assert api.device_status() == 1  # NVQ_ERR_INVALID
    check_decode(o, lse, ref, 300, vmax)
    # a length over the table's: only the table's pages
    o, lse = api.attn_qat_cross(args[0][:70], args[1], args[2][:1, 1:].contiguous(), ints([100000]),
                                scale=0.125)
    assert api.device_status() == 1
    ref = os_.attend(q[:70], pool, [(table[0, 1:].clamp(0, pages - 1), 256)], 0.125)
    if int(table[0, 2]) < pages:
        check_decode(o, lse, ref, 256, vmax)
    # offsets beyond the rows, or decreasing: cut
    for bad in ([0, 70, 71, 1 << 30], [-5, 70, 71, 90], [0, 70, 30, 90]):
        api.attn_qat_cross(*args, ints(bad), 0.125)
        assert api.device_status() == 1
    good = os_.attend(q[:10], pool, [(table[0, 1:2], 128)], 0.125)
    o, lse = api.attn_qat_cross(args[0], args[1], args[2][:1, 1:2].contiguous(), ints([128]),
                                ints([-4, 10]), 0.125)
    assert api.device_status() == 1
    check_decode(o[:10], lse[:10], good, 128, vmax)
    assert not bool(o[10:].any()) and bool((lse[10:] == -float("inf")).all())


def test_no_keys_no_rows():
    pool = torch.full((2, 2, 144 * 64), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    q = torch.randn(40, 4, 64, device="cuda").to(BF16)
    lens = ints([0, 0, -4, 0, 0])
    o, lse = api.attn_qat_cross(q, pool, table, lens, ints([0, 3, 3, 30, 31, 35]))
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    o, lse = api.attn_qat_cross(q, pool, table, lens + 200, ints([7] * 6))  # no sequence has rows
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    o, lse = api.attn_qat_cross(q[:0], pool, table, lens, ints([0] * 6))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = api.attn_qat_cross(q, pool, table[:0], lens[:0], ints([0]))
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    o, lse = api.attn_qat_decode_prefix(q[:5], pool, table, lens, table[:2], lens[:2], ints([0, 2, 5]))
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    o, lse = api.attn_qat_decode_prefix(q[:0], pool, table[:0], lens[:0], table[:2], lens[:2],
                                        ints([0, 0, 0]))
    assert o.shape == (0, 4, 64) and api.device_status() == 0


PREFIXES = [  # h, hkv, d, sequences and prefix of each group, own lengths, sequences in front, behind
    (1, 1, 128, [(1, 1)], [1], 0, 0), (4, 4, 64, [(3, 500)], [0, 1, 129], 0, 0),
    (8, 2, 128, [(5, 1000)], [128, 0, 300, 7, 64], 0, 0),
    (8, 2, 64, [(2, 300), (3, 0), (4, 128)], [5, 0, 0, 200, 1, 3, 0, 128, 300], 0, 0),
    (24, 2, 128, [(3, 129), (2, 127)], [5, 0, 200, 1, 3, 70, 0], 1, 1),
    (16, 1, 64, [(20, 2100)], [i * 7 for i in range(20)], 0, 0),
    (12, 12, 128, [(2, 777), (0, 300), (1, 40)], [30, 200, 5, 9], 0, 1),
]


@pytest.mark.parametrize("case", PREFIXES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}_{len(c[3])}_{c[3][0][1]}")
def test_decode_prefix_parity(case):
    h, hkv, d, groups, own, front, behind = case
    g = torch.Generator().manual_seed(h * d + len(own))
    shared = [n for _, n in groups]
    table, pages = tables(own + shared, max(-(-max(own + shared) // PAGE), 1) + 1, g)
    pool = make_pool(pages, hkv, d, g)
    vmax = vmax_of(pool, d)
    spoil(pool, table, own + shared, d)
    b = len(own)
    cu = offsets([n for n, _ in groups], front)
    assert cu[-1] + behind == b
    q = queries(b, h, d, g)
    prefix, mine = table[b:], table[:b]
    refs = []
    for i in range(b):
        s = [x for x in range(len(groups)) if cu[x] <= i < cu[x + 1]]
        spans = [(prefix[x], shared[x]) for x in s] + [(mine[i], own[i])]
        refs.append(os_.attend(q[i:i + 1], pool, spans, d ** -0.5))
    ref = tuple(torch.cat(x) for x in zip(*refs))
    ws = torch.full((api.attn_qat_decode_prefix_workspace(b, len(groups), h, hkv, d, mine.shape[1],
                                                          prefix.shape[1]),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    args = (q.cuda(), pool.cuda(), mine.cuda(), ints(own), prefix.cuda(), ints(shared))
    o, lse = api.attn_qat_decode_prefix(*args, ints(cu), workspace=ws)
    assert api.device_status() == 0
    check_decode(o, lse, ref, max(own) + max(shared), vmax)
    o2, lse2 = api.attn_qat_decode_prefix(*args, ints(cu), workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if len(groups) == 1:
        o2, lse2 = api.attn_qat_decode_prefix(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_prefix_of_many_sequences_is_the_decode_over_both():
    """Groups of many, own keys long and short: within the bounds that both calls keep, the decode
    whose tables hold the prefix's pages in front (prefixes of whole pages)."""
    h, hkv, d, b = 8, 2, 128, 150
    g = torch.Generator().manual_seed(21)
    pool = make_pool(60, hkv, d, g).cuda()
    prefix = torch.randint(0, 60, (3, 30), generator=g).int()
    pages = [30, 11, 0]
    own = torch.randint(0, 2500, (b,), generator=g)
    own[::9] = 0
    mine = torch.randint(0, 60, (b, 20), generator=g).int()
    cu = [0, 80, 149, 150]
    both = torch.zeros(b, 50, dtype=torch.int32)
    total = own.clone()
    for s in range(3):
        for i in range(cu[s], cu[s + 1]):
            both[i, :pages[s]], both[i, pages[s]:pages[s] + 20] = prefix[s, :pages[s]], mine[i]
            total[i] += pages[s] * PAGE
    q = torch.randn(b, h, d, generator=g).to(BF16).cuda()
    o, lse = api.attn_qat_decode_prefix(q, pool, mine.cuda(), own.int().cuda(), prefix.cuda(),
                                        ints([n * PAGE for n in pages]), ints(cu))
    o2, lse2 = api.attn_qat_decode(q, pool, both.cuda(), total.int().cuda())
    keys = total[:, None, None] > 0
    # both sides' bounds: a bf16 step between neighbours; of values up to vmax twice the share of
    # p in f16; the sums of S, with scale sum |q k| below 16, 2 vmax 16 2^-16 a side
    vmax = vmax_of(pool, d)
    tol = o2.cpu().double().abs() * 2.0 ** -7 + 2 * vmax * (2.0 ** -11 + 2.0 ** -12) + \
        vmax * 2.0 ** -10
    assert bool((((o.cpu().double() - o2.cpu().double()).abs() <= tol) | ~keys).all())
    fin = torch.isfinite(lse2)
    assert torch.equal(torch.isfinite(lse), fin)
    assert bool(((lse - lse2)[fin].abs() <= 2.0 ** -11).all()) and api.device_status() == 0


@pytest.mark.parametrize("own", [0, 5, 300])
def test_a_nan_in_a_cached_key_is_seen(own):
    """A NaN scale byte among the keys: rows that see it are NaN, others as they were; also where
    the prefix holds it and the sequence's own keys are none, few, or cut into parts."""
    h, hkv, d = 4, 2, 128
    g = torch.Generator().manual_seed(own)
    pool = make_pool(8, hkv, d, g)
    pool[1, 1, 128 * d + 7 * d // 16] = 0x7F  # K's scales, page 1, head 1, key 7
    q = torch.randn(4, h, d, generator=g).to(BF16).cuda()
    prefix, shared = ints([[0, 1], [2, 3]]), ints([200, 200])
    table, lens = ints([[4, 5, 6]] * 4), ints([own] * 4)
    pool = pool.cuda()
    o, _ = api.attn_qat_decode_prefix(q, pool, table, lens, prefix, shared)
    sees = torch.zeros(4, h, dtype=torch.bool)
    sees[:2, 2:] = True
    assert torch.equal(o.isnan().all(-1).cpu(), sees) and torch.equal(o.isnan().any(-1).cpu(), sees)
    o, lse = api.attn_qat_cross(q, pool, prefix, shared)
    assert torch.equal(o.isnan().all(-1).cpu(), sees) and torch.equal(o.isnan().any(-1).cpu(), sees)
    assert bool(torch.isfinite(lse.cpu()[~sees]).all()) and api.device_status() == 0


def test_offsets_past_32_bits():
    """A pool of over 4 GiB: pages at its end, read where they are."""
    hkv, d = 8, 128
    pages = (1 << 32) // (hkv * 144 * d) + 40
    g = torch.Generator().manual_seed(8)
    small = make_pool(2, hkv, d, g).cuda()
    pool = torch.zeros(pages, hkv, 144 * d, dtype=torch.uint8, device="cuda")
    pool[-2:] = small
    q = torch.randn(50, 16, d, generator=g).to(BF16).cuda()
    table, lens = ints([[pages - 1, pages - 2]]), ints([200])
    o, lse = api.attn_qat_cross(q, pool, table, lens)
    o2, lse2 = api.attn_qat_cross(q, small, table - (pages - 2), lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    own = ints([[pages - 2]] * 50)
    o, lse = api.attn_qat_decode_prefix(q, pool, own, lens.expand(50).contiguous() - 100, table, lens)
    o2, lse2 = api.attn_qat_decode_prefix(q, small, own - (pages - 2),
                                          lens.expand(50).contiguous() - 100, table - (pages - 2), lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and api.device_status() == 0


def test_graphs_share_a_workspace_and_follow_lengths():
    d, hkv, h, b = 128, 2, 8, 6
    g = torch.Generator().manual_seed(13)
    pool = make_pool(60, hkv, d, g).cuda()
    table = torch.randperm(60, generator=g).int().view(b, 10).cuda()
    lens, shared = ints([5, 900, 130, 0, 7, 1280]), ints([700, 128])
    cu = ints([0, 4, 6])
    prefix = table[:2].flip(1).contiguous()
    qs = [torch.randn(b, h, d, generator=g).to(BF16).cuda() for _ in range(2)]
    calls = [lambda q, **k: api.attn_qat_decode_prefix(q, pool, table, lens, prefix, shared, cu, **k),
             lambda q, **k: api.attn_qat_cross(q, pool, prefix, shared, cu, **k)]
    ws = torch.empty(api.attn_qat_decode_prefix_workspace(b, 2, h, hkv, d, 10, 10),
                     dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(b, h, device="cuda")) for q in qs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for q, call, (o, l) in zip(qs, calls, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(q, o=o, lse=l, workspace=ws)
        graphs.append(graph)
    for step, pre, off in (([5, 900, 130, 0, 7, 1280], [700, 128], [0, 4, 6]),
                           ([129, 0, 1, 5, 5, 5], [0, 1280], [0, 1, 5]),
                           ([0] * 6, [1, 1000], [2, 2, 6])):
        for t, v in ((lens, step), (shared, pre), (cu, off)):
            t.copy_(torch.tensor(v, dtype=torch.int32))
        for graph in graphs + graphs:
            graph.replay()
        torch.cuda.synchronize()
        for q, call, (o, l) in zip(qs, calls, outs):
            o2, l2 = call(q)
            assert torch.equal(o, o2) and torch.equal(l, l2)
    assert api.device_status() == 0


def test_two_streams_at_once():
    d, hkv, h = 64, 4, 8
    g = torch.Generator().manual_seed(14)
    pool = make_pool(200, hkv, d, g).cuda()
    table = torch.randperm(200, generator=g).int().view(4, 50).cuda()
    lens = ints([6400, 600, 100, 3000])
    qs = [torch.randn(400, h, d, generator=g).to(BF16).cuda() for _ in range(2)]
    calls = [lambda q: api.attn_qat_cross(q, pool, table, lens),
             lambda q: api.attn_qat_decode_prefix(q[:4], pool, table, lens, table[:1], lens[:1])]
    want = [call(q)[0] for q, call in zip(qs, calls)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i](qs[i])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])
    assert api.device_status() == 0


def test_refusals_on_device_tensors():
    pool = torch.zeros(4, 2, 144 * 64, dtype=torch.uint8, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = ints([1, 1])
    q = torch.zeros(4, 4, 64, dtype=BF16, device="cuda")
    for bad in (dict(q=q[:3]), dict(q=q.float()), dict(pool=pool[:, :, :-16]), dict(lens=lens.long()),
                dict(table=table.t()), dict(lens=lens[:1]), dict(pool=pool.cpu()), dict(cu=lens),
                dict(q=q.transpose(1, 2)), dict(o=q[:, :2]), dict(lse=lens),
                dict(workspace=torch.zeros(1, device="cuda").expand(1 << 26))):
        a = dict(q=q, pool=pool, table=table, lens=lens) | bad
        more = {n: a[n] for n in ("o", "lse", "workspace") if n in a}
        with pytest.raises(ValueError):
            api.attn_qat_cross(a["q"], a["pool"], a["table"], a["lens"], a.get("cu"), **more)
        if "q" in bad:
            continue
        with pytest.raises(ValueError):
            api.attn_qat_decode_prefix(q[:2], a["pool"], a["table"], a["lens"], table, lens,
                                       a.get("cu"), **more)
        if "pool" not in bad and "cu" not in bad and not more:
            with pytest.raises(ValueError):
                api.attn_qat_decode_prefix(q[:2], pool, table, lens, a["table"], a["lens"])
    with pytest.raises(ValueError):
        api.attn_qat_decode_prefix(q[:3], pool, table, lens, table, lens)  # 3 rows, 2 sequences
    with pytest.raises(ValueError):
        api.attn_qat_decode_prefix(q[:2], pool, table, lens, table.repeat(2, 1)[:3], lens.repeat(2)[:3])
    with pytest.raises(api._lib.NvqError):
        api.attn_qat_cross(q[:, :3].contiguous(), pool, table, lens)  # 3 heads over 2
    with pytest.raises(api._lib.NvqError):
        api.attn_qat_cross(q, pool, table, lens, o=q)  # over its queries
    small = torch.empty(256, dtype=torch.uint8, device="cuda")  # too small: one of the call's own
    assert torch.equal(api.attn_qat_cross(q, pool, table, lens, workspace=small)[0],
                       api.attn_qat_cross(q, pool, table, lens)[0])


def test_outputs_given_are_marked_as_written():
    pool, table = api.nvfp4_kv_pool(1, 1, 64), ints([[0]])
    q = torch.randn(3, 2, 64, device="cuda").to(BF16)
    for call in (lambda o: api.attn_qat_cross(q, pool, table, ints([9]), o=o),
                 lambda o: api.attn_qat_decode_prefix(q, pool, table.expand(3, 1).contiguous(),
                                                      ints([1, 1, 1]), table, ints([4]), o=o)):
        o = torch.zeros(3, 2, 64, dtype=BF16, device="cuda")
        y = (torch.ones((), device="cuda", requires_grad=True).to(BF16) * o).sum()
        call(o)
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
