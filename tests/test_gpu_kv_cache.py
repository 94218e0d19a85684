"""The paged NVFP4 cache on the GPU against oracle/serving.py.

Append: code and scale bytes equal the oracle's; every byte of the pool that no new token
owns stays as it was.

Decode: per element of o, with A = sum p |v| / l and E = scale max_j sum |q k_j| of the
float64 oracle,
  2^-8 |o|                          the bf16 rounding of the result
  + A (2^-11 + 2^-12)               p rounded to f16, the fp32 exponentials and sums
  + n 2^-25 max |v|                 p below f16's normal range (n visible keys)
  + 2 A E 128 2^-23                 S: exact products, up to 128 fp32 additions of truncated
                                    half a step, twice for the exponential's slope and l's
and lse is within E 128 2^-23 + 2^-20 + |lse| 2^-23 of the oracle's.
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_

pytestmark = pytest.mark.gpu
BF16, PAGE = torch.bfloat16, 128


def make_pool(pages, hkv, d, g):
    """A pool of random tokens with stale garbage (NaN scale bytes among it) nowhere yet."""
    pool = torch.empty(pages, hkv, 144 * d, dtype=torch.uint8)
    for at_c, at_s in ((0, 128 * d), (64 * d, 136 * d)):
        x = torch.randn(pages, hkv, PAGE, d, generator=g)
        x[..., :3] *= 6  # larger channels
        c, s = os_.pack(x.to(BF16))
        pool[:, :, at_c:at_c + 64 * d] = c.flatten(2)
        pool[:, :, at_s:at_s + 8 * d] = s.flatten(2)
    return pool


def spoil(pool, table, lens, d):
    """NaN scale bytes and arbitrary codes in the rows behind each sequence's last token."""
    for i, n in enumerate(lens):
        if n > 0 and n % PAGE:
            p, r = int(table[i, n // PAGE]), n % PAGE
            for at, w, v in ((0, d // 2, 0xFF), (64 * d, d // 2, 0x77), (128 * d, d // 16, 0x7F),
                             (136 * d, d // 16, 0xFF)):
                pool[p, :, at + r * w:at + PAGE * w] = v


def tables(lens, capacity, g, extra=2):
    need = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(sum(need) + extra, generator=g).int()
    table = torch.full((len(lens), capacity), 1 << 30, dtype=torch.int32)  # unread entries
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + extra


def check_decode(o, lse, ref, n_max, vmax):
    r, l, mag, e = ref
    es = e[..., None] * 2.0 ** -16
    tol = r.abs() * 2.0 ** -8 + mag * (2.0 ** -11 + 2.0 ** -12) + n_max * 2.0 ** -25 * vmax + \
        2 * mag * es
    err = (o.cpu().double() - r).abs()
    assert bool((err <= tol).all()), (float((err / tol.clamp_min(1e-30)).max()), float(err.max()))
    lse = lse.cpu().double()
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    el = (lse - l)[~empty].abs()
    assert bool((el <= es[..., 0][~empty] + 2.0 ** -20 + l[~empty].abs() * 2.0 ** -23).all()), \
        float(el.max())


CASES = [  # h, hkv, d, window, sinks, lengths
    (1, 1, 128, 0, 0, [1]),
    (4, 4, 64, 0, 0, [128, 1, 0, 127, 129]),
    (8, 2, 128, 0, 0, [300, 5, 641]),
    (7, 1, 128, 0, 0, [1000, 0]),
    (12, 12, 128, 0, 0, [777]),
    (16, 1, 64, 0, 0, [2000, 17, 256]),
    (24, 2, 64, 0, 0, [383, 384, 385]),
    (40, 1, 128, 0, 0, [130, 64]),
    (6, 2, 128, 1, 0, [1, 2, 128, 129, 500]),
    (6, 2, 128, 100, 4, [3, 99, 104, 105, 128, 228, 700]),
    (4, 2, 64, 128, 1, [128, 129, 256, 257, 900]),
    (4, 1, 64, 5, 200, [190, 206, 700, 0]),
    (2, 1, 128, 4096, 4, [5000, 70]),
    (2, 2, 64, 130, 129, [255, 260, 1025]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}_w{c[3]}s{c[4]}_{c[5][0]}")
def test_decode_parity(case):
    h, hkv, d, window, sinks, lens = case
    g = torch.Generator().manual_seed(sum(lens) + h)
    table, pages = tables(lens, -(-max(lens) // PAGE) + 2, g)
    pool = make_pool(pages, hkv, d, g)
    vmax = float(os_.unpack(*os_.record_parts(pool, d)[1::2]).abs().max())
    spoil(pool, table, lens, d)
    b = len(lens)
    qbuf = torch.randn(b, h * d + 16, generator=g).to(BF16).cuda()
    q = qbuf[:, :h * d].view(b, h, d)  # strided rows
    lens_t = torch.tensor(lens, dtype=torch.int32)
    scale = d ** -0.5
    ref = os_.decode(q.cpu(), pool, table, lens, scale, window, sinks)
    # a workspace of arbitrary bytes (NaN patterns), the second call on the first's
    ws = torch.full((api.attn_qat_decode_workspace(b, h, hkv, d, table.shape[1]),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    args = (q, pool.cuda(), table.cuda(), lens_t.cuda(), scale, window, sinks)
    o, lse = api.attn_qat_decode(*args, workspace=ws)
    check_decode(o, lse, ref, max(lens), vmax)
    o2, lse2 = api.attn_qat_decode(*args, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert api.device_status() == 0


@pytest.mark.parametrize("h,hkv,d,b,longest,window,sinks", [
    (2, 1, 64, 700, 400, 0, 0), (32, 2, 128, 200, 600, 0, 0), (4, 4, 128, 150, 900, 200, 3),
    (18, 2, 64, 180, 300, 0, 0), (4, 2, 64, 400, 700, 0, 0), (5, 1, 64, 70, 7000, 0, 0)])
def test_decode_of_many_sequences(h, hkv, d, b, longest, window, sinks):
    """More segments than the chip has runs, some sequences empty, pages shared between
    sequences, the table a slice of a wider one."""
    g = torch.Generator().manual_seed(b + h)
    lens = torch.randint(0, longest + 1, (b,), generator=g, dtype=torch.int32)
    lens[torch.rand(b, generator=g) < 0.1] = 0
    lens[b // 2] = longest
    pages, width = 40, -(-longest // PAGE)
    pool = make_pool(pages, hkv, d, g)
    vmax = float(os_.unpack(*os_.record_parts(pool, d)[1::2]).abs().max())
    wide = torch.randint(0, pages, (b, width + 3), generator=g, dtype=torch.int32)
    q = torch.randn(b, h, d, generator=g).to(BF16)
    ref = os_.decode(q, pool, wide[:, :width], lens.tolist(), d ** -0.5, window, sinks)
    args = (q.cuda(), pool.cuda(), wide.cuda()[:, :width], lens.cuda(), d ** -0.5, window, sinks)
    o, lse = api.attn_qat_decode(*args)
    check_decode(o, lse, ref, longest, vmax)
    o2, lse2 = api.attn_qat_decode(*args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert api.device_status() == 0


def test_decode_of_empty_sequences_only():
    pool = torch.full((2, 2, 144 * 64), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 0, -4, 0, 0], dtype=torch.int32, device="cuda")
    q = torch.randn(5, 4, 64, device="cuda").to(BF16)
    o, lse = api.attn_qat_decode(q, pool, table, lens)
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    assert api.device_status() == 0


def test_sharp_scores_and_negative_sums():
    """Scores hundreds apart (all weight on one key, anywhere in the sequence) and all far
    below zero: the running maximum and the join must not lose either."""
    d, n = 64, 1500
    g = torch.Generator().manual_seed(3)
    table, pages = tables([n] * 4, 12, g)
    pool = make_pool(pages, 1, d, g)
    q = torch.randn(4, 2, d, generator=g).to(BF16)
    for scale in (30.0, 1e-3):
        ref = os_.decode(q, pool, table, [n] * 4, scale)
        o, lse = api.attn_qat_decode(q.cuda(), pool.cuda(), table.cuda(),
                                     torch.full((4,), n, dtype=torch.int32, device="cuda"), scale)
        vmax = float(os_.unpack(*os_.record_parts(pool, d)[1::2]).abs().max())
        check_decode(o, lse, ref, n, vmax)
    assert api.device_status() == 0


def test_bad_pages_and_lengths_are_left_out_and_reported():
    d, lens = 64, [300, 200, 130]
    g = torch.Generator().manual_seed(4)
    table, pages = tables(lens, 3, g)
    pool = make_pool(pages, 2, d, g)
    vmax = float(os_.unpack(*os_.record_parts(pool, d)[1::2]).abs().max())
    table[0, 1], table[1, 0] = -1, pages  # one page past the pool's end, one negative
    q = torch.randn(3, 4, d, generator=g).to(BF16)
    gone = {(0, 1), (1, 0)}
    ref = os_.decode(q, pool, table.clamp(0, pages - 1), lens, 0.125,
                     keep=lambda b, j: (b, j // PAGE) not in gone)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = api.attn_qat_decode(q.cuda(), pool.cuda(), table.cuda(), lens_t, 0.125)
    assert api.device_status() == 1  # NVQ_ERR_INVALID
    check_decode(o, lse, ref, 300, vmax)
    assert api.device_status() == 0
    # a length over the table's: only the table's pages
    ref = os_.decode(q[2:], pool, table[2:], [256], 0.125)
    pool_c = pool.cuda()
    o, lse = api.attn_qat_decode(q[2:].cuda(), pool_c, table[2:, :2].contiguous().cuda(),
                                 torch.tensor([100000], dtype=torch.int32, device="cuda"), 0.125)
    assert api.device_status() == 1
    check_decode(o, lse, ref, 256, vmax)
    # append: the bad tokens are not written, the others are
    k = torch.randn(3, 2, d, generator=g).to(BF16).cuda()
    before = pool_c.clone()
    table[1, 1] = -5  # position 199
    api.nvfp4_kv_append(k, k, torch.tensor([900, 200, -4], dtype=torch.int32, device="cuda"),
                        table.cuda(), pool_c)
    assert api.device_status() == 1 and torch.equal(pool_c, before)


APPENDS = [  # hkv, d, (new, before) per sequence, single-token form
    (1, 64, [(1, 0)], True), (3, 128, [(1, 127), (1, 128), (1, -1), (1, 300)], True),
    (2, 128, [(5, 0), (0, 10), (300, 100), (1, 255)], False), (5, 64, [(130, 0)], False),
    (12, 128, [(17, 120)], False), (2, 64, [(1, i) for i in range(70)], True),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{c[0]}x{c[1]}_{len(c[2])}_{c[2][0]}")
def test_append_is_bit_exact_and_touches_nothing_else(case):
    hkv, d, runs, single = case
    g = torch.Generator().manual_seed(len(runs) * 7 + d)
    lens = [n + b for n, b in runs]
    table, pages = tables(lens, -(-max(lens) // PAGE) + 1, g)
    t = sum(n for n, _ in runs)
    pad = 0 if single else 4  # rows behind the last sequence
    kv = torch.randn(t + pad, 2 * hkv * d + 8, generator=g).to(BF16)
    kv[:, ::5] *= 50
    kv[0, :32] = 0.0
    kv[0, 3] = -0.0
    kv[-1 - pad, :16] = 2.0 ** -126
    kv = kv.cuda()
    k, v = kv[:, :hkv * d].view(-1, hkv, d), kv[:, 8 + hkv * d:].view(-1, hkv, d)
    pool = torch.randint(0, 256, (pages, hkv, 144 * d), generator=g).to(torch.uint8)
    want = pool.clone()
    cu, at = [0], 0
    for (n, before), i in zip(runs, range(len(runs))):
        for j in range(n):
            pos = before + j
            if before < 0:
                continue
            p, r = int(table[i, pos // PAGE]), pos % PAGE
            for x, at_c, at_s in ((k, 0, 128 * d), (v, 64 * d, 136 * d)):
                c, s = os_.pack(x[at + j].cpu())
                want[p, :, at_c + r * d // 2:at_c + (r + 1) * d // 2] = c
                want[p, :, at_s + r * d // 16:at_s + (r + 1) * d // 16] = s
        at += n
        cu.append(at)
    pool = pool.cuda()
    api.nvfp4_kv_append(k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), table.cuda(),
                        pool, None if single else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert api.device_status() == 0
    assert torch.equal(pool.cpu(), want)


def test_offsets_past_32_bits():
    """A pool of over 4 GiB: the last page is written and read where it is."""
    hkv, d = 8, 128
    pages = (1 << 32) // (hkv * 144 * d) + 40
    pool = torch.zeros(pages, hkv, 144 * d, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(140, hkv, d, generator=g).to(BF16).cuda() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([140], dtype=torch.int32, device="cuda")
    api.nvfp4_kv_append(k, v, lens, table, pool, torch.tensor([0, 140], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 16, d, generator=g).to(BF16).cuda()
    o, lse = api.attn_qat_decode(q, pool, table, lens)
    small = pool[-2:].clone()
    o2, lse2 = api.attn_qat_decode(q, small, table - (pages - 2), lens)
    assert api.device_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert not bool(pool[:-2].any())
    ref = os_.decode(q.cpu(), small.cpu(), torch.tensor([[1, 0]]), [140], d ** -0.5)
    check_decode(o, lse, ref, 140, 8.0)


def test_long_sequence_sampled_against_its_own_windows():
    """One long sequence next to short ones: the split result equals the join, by the
    operator's own log-sum-exp, of decodes over table slices of the same cache."""
    d, hkv, h, n = 128, 2, 6, 40000
    g = torch.Generator().manual_seed(12)
    pages = -(-n // PAGE)
    pool = make_pool(64, hkv, d, g).cuda()  # pages reused: 64 distinct ones
    table = torch.randint(0, 64, (3, pages), generator=g).int().cuda()
    lens = torch.tensor([n, 3, 500], dtype=torch.int32, device="cuda")
    q = torch.randn(3, h, d, generator=g).to(BF16).cuda()
    o, lse = api.attn_qat_decode(q, pool, table, lens)
    parts = []
    for p0 in range(0, pages, 50):
        m = min(50, pages - p0)
        ln = torch.tensor([min(n - p0 * PAGE, m * PAGE)], dtype=torch.int32, device="cuda")
        parts.append(api.attn_qat_decode(q[:1], pool, table[:1, p0:p0 + m].contiguous(), ln))
    ls = torch.stack([p[1][0].double() for p in parts])
    w = torch.softmax(ls, 0)
    want = sum(w[i][:, None] * parts[i][0][0].double() for i in range(len(parts)))
    # both sides carry a bf16 rounding (2^-8 of each part's |o|) and the f16 p
    mag = sum(w[i][:, None] * parts[i][0][0].double().abs() for i in range(len(parts)))
    tol = (want.abs() + mag) * 2.0 ** -8 + 2.0 ** -9
    assert bool(((o[0].double() - want).abs() <= tol).all())
    assert bool(((lse[0].double() - torch.logsumexp(ls, 0)).abs() <= 2.0 ** -14).all())
    assert api.device_status() == 0


def test_replayed_graphs_share_a_workspace_and_follow_lengths():
    d, hkv, h, b = 128, 2, 8, 3
    g = torch.Generator().manual_seed(13)
    pool = make_pool(30, hkv, d, g).cuda()
    table = torch.randperm(30, generator=g).int().view(b, 10).cuda()
    lens = torch.tensor([5, 900, 130], dtype=torch.int32, device="cuda")
    qs = [torch.randn(b, h, d, generator=g).to(BF16).cuda() for _ in range(2)]
    kv = torch.randn(b, hkv, d, generator=g).to(BF16).cuda()
    ws = torch.empty(api.attn_qat_decode_workspace(b, h, hkv, d, 10), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty(b, h, device="cuda")) for q in qs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for q, (o, l) in zip(qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            api.nvfp4_kv_append(kv, kv, lens, table, pool)
            api.attn_qat_decode(q, pool, table, lens, workspace=ws, o=o, lse=l)
        graphs.append(graph)
    for step in ([5, 900, 130], [129, 1280, 1], [0, 257, 640]):
        lens.copy_(torch.tensor(step, dtype=torch.int32))
        for graph in graphs + graphs:
            graph.replay()
        torch.cuda.synchronize()
        for q, (o, l) in zip(qs, outs):
            o2, l2 = api.attn_qat_decode(q, pool, table, lens)
            assert torch.equal(o, o2) and torch.equal(l, l2)
    assert api.device_status() == 0


def test_two_streams_at_once():
    d, hkv, h = 64, 4, 8
    g = torch.Generator().manual_seed(14)
    pool = make_pool(200, hkv, d, g).cuda()
    table = torch.randperm(200, generator=g).int().view(4, 50).cuda()
    lens = torch.tensor([6400, 6000, 100, 3000], dtype=torch.int32, device="cuda")
    qs = [torch.randn(4, h, d, generator=g).to(BF16).cuda() for _ in range(2)]
    want = [api.attn_qat_decode(q, pool, table, lens)[0] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(api.attn_qat_decode(qs[i], pool, table, lens)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


def test_refusals_on_device_tensors():
    pool = torch.zeros(4, 2, 144 * 64, dtype=torch.uint8, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=BF16, device="cuda")
    for bad in (dict(q=q[:1]), dict(q=q.float()), dict(pool=pool[:, :, :-16]), dict(lens=lens.long()),
                dict(table=table.t()), dict(lens=lens[:1]), dict(pool=pool.cpu()),
                dict(q=q.transpose(1, 2))):
        a = dict(q=q, pool=pool, table=table, lens=lens) | bad
        with pytest.raises(ValueError):
            api.attn_qat_decode(a["q"], a["pool"], a["table"], a["lens"])
    with pytest.raises(api._lib.NvqError):
        api.attn_qat_decode(q[:, :3].contiguous(), pool, table, lens)  # 3 heads over 2
    for bad in (dict(v=k[:1]), dict(k=k[:, :1].contiguous(), v=k[:, :1].contiguous()),
                dict(cu=lens), dict(k=torch.cat((k, k)), v=torch.cat((k, k)))):
        a = dict(k=k, v=k, cu=None) | bad
        with pytest.raises(ValueError):
            api.nvfp4_kv_append(a["k"], a["v"], lens, table, pool, a["cu"])
