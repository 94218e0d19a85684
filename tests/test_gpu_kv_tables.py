"""The cache's tables on the GPU (nvfp4_kv_extend, nvfp4_kv_release, nvfp4_kv_append_slots)
against oracle/serving.py: every value equal, and nothing else written."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_

pytestmark = pytest.mark.gpu
I32, PAGE = torch.int32, 128


def ints(values, dtype=I32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def state(lens, wide, spare, seed, guard=True):
    """(table as lists, free pages, pages): random pages, entries of no page -7."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // PAGE) for n in lens]
    pages = sum(need) + spare + 2
    perm = torch.randperm(pages, generator=g).tolist()
    table, at = [], 0
    for n in need:
        table.append(perm[at:at + n] + [-7] * (wide - n))
        at += n
    return table, perm[at:at + spare], pages


def run_extend(new, lens, table, free, pages, tokens, start=None, **outs):
    padded = free + [-9] * (pages - len(free))
    args = ints(new), ints(lens), ints(table), ints(padded), ints([len(free)])
    got = api.nvfp4_kv_extend(*args, tokens=tokens, start=None if start is None else ints(start),
                              **outs)
    return got, args


def check(got, args, want):
    after, left, cu, positions, slots, table = want
    assert got.seq_lens.tolist() == after and got.free_count.tolist() == [left]
    assert got.cu_tokens.tolist() == cu
    assert torch.equal(got.positions, ints(positions)) and got.slots.dtype == torch.int64
    assert torch.equal(got.slots, ints(slots, torch.int64))
    assert torch.equal(args[2], ints(table))


CASES = [  # new tokens, tokens held
    ([1], [0]), ([0], [0]), ([0, 0, 0], [5, 0, 300]), ([1, 1, 1, 1], [127, 128, 129, 0]),
    ([-3, 2, 1], [10, -4, 255]), ([128, 129, 127, 1, 0], [0, 0, 1, 127, 128]),
    ([700, 1, 0, 300], [60, 1000, 5, 0]), ([5000], [1]), ([2047, 1], [0, 128]),
    ([2048, 1], [0, 128]), ([9000, 0, 4000, 77], [130, 7, 0, 255]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}_{c[0][0]}_{c[1][0]}")
@pytest.mark.parametrize("extra", [0, 5, 3000])
def test_extend(case, extra):
    new, lens = case
    wide = max(-(-(max(t, 0) + max(n, 0)) // PAGE) for t, n in zip(new, lens)) + 1
    grown = sum(-(-(max(t, 0) + max(n, 0)) // PAGE) - -(-max(n, 0) // PAGE)
                for t, n in zip(new, lens))
    table, free, pages = state(lens, wide, grown + extra % 7, seed=len(new) + extra)
    tokens = sum(max(t, 0) for t in new) + extra
    start = [1000 * i - 500 for i in range(len(new))] if extra else None
    got, args = run_extend(new, lens, table, free, pages, tokens, start)
    check(got, args, os_.extend(new, lens, table, free, len(free), tokens, start))
    assert args[3].tolist() == free + [-9] * (pages - len(free))  # the stack itself stays
    assert api.device_status() == 0
    again = api.nvfp4_kv_extend(*args, tokens=tokens, start=None if start is None else ints(start))
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("b,most,seed", [(1000, 3, 0), (1024, 300, 1), (1025, 5, 2), (3000, 140, 3),
                                         (65535, 2, 4)])
def test_extend_of_many_sequences(b, most, seed):
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(0, most, (b,), generator=g).tolist()
    lens = torch.randint(0, 400, (b,), generator=g).tolist()
    table, free, pages = state(lens, 6, b + most * b // PAGE + 1, seed)
    tokens = sum(new) + 3
    got, args = run_extend(new, lens, table, free, pages, tokens)
    check(got, args, os_.extend(new, lens, table, free, len(free), tokens))
    assert api.device_status() == 0


def test_extend_where_nothing_fits_changes_nothing():
    """Too few pages, rows or table columns, a count out of range: all or nothing."""
    new, lens = [200, 1, 4], [100, 128, 0]
    table, free, pages = state(lens, 4, 4, seed=9)
    fits = dict(new=new, lens=lens, table=table, free=free, pages=pages, tokens=205)
    assert os_.extend(new, lens, table, free, 4, 205) is not None
    for bad in (dict(free=free[:3]), dict(free=[]), dict(tokens=204), dict(tokens=0),
                dict(new=[500, 1, 4], tokens=600), dict(lens=[100, 128, 1 << 30]),
                dict(lens=[100, 2 ** 31 - 1, 0]), dict(new=[2 ** 31 - 1, 2 ** 31 - 1, 4])):
        a = fits | bad
        for tokens in {a["tokens"], max(a["tokens"], 4000) if "free" in bad else a["tokens"]}:
            got, args = run_extend(a["new"], a["lens"], a["table"], a["free"], a["pages"], tokens)
            assert got.seq_lens.tolist() == a["lens"]
            assert got.free_count.tolist() == [len(a["free"])]
            assert got.cu_tokens.tolist() == [0] * 4
            assert bool((got.positions == -1).all()) and bool((got.slots == -1).all())
            assert args[2].tolist() == a["table"]
            assert api.device_status() == 1 and api.device_status() == 0
    for count in (-1, pages + 1, 2 ** 31 - 1):
        args = (ints(new), ints(lens), ints(table), ints(free + [-9] * (pages - 4)), ints([count]))
        got = api.nvfp4_kv_extend(*args, tokens=205)
        assert got.free_count.tolist() == [count] and not bool(got.cu_tokens.any())
        assert api.device_status() == 1


def test_extend_reports_a_page_outside_the_pool():
    got, args = run_extend([1, 1, 1], [5, 5, 0], [[-1, -7], [99, -7], [-7, -7]], [1000], 12, 3)
    assert got.slots.tolist() == [-1, -1, -1] and got.positions.tolist() == [5, 5, 0]
    assert args[2].tolist() == [[-1, -7], [99, -7], [1000, -7]]
    assert api.device_status() == 1


def test_extend_in_place_in_a_graph():
    """A captured step advances lengths and free pages in place; replays follow the changes that
    the host makes between them."""
    lens, new = [126, 0, 300, 5], [1, 1, 0, 1]
    table, free, pages = state(lens, 5, 6, seed=3)
    dl, dn, dt, df, dc = ints(lens), ints(new), ints(table), ints(free + [-9] * (pages - 6)), ints([6])
    outs = dict(seq_lens_out=dl, free_count_out=dc, cu_tokens=ints([0] * 5),
                positions=ints([0] * 6), slots=ints([0] * 6, torch.int64))
    saved = [t.clone() for t in (dl, dt, dc)]
    api.nvfp4_kv_extend(dn, dl, dt, df, dc, tokens=6, **outs)  # warm-up
    for t, v in zip((dl, dt, dc), saved):
        t.copy_(v)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        api.nvfp4_kv_extend(dn, dl, dt, df, dc, tokens=6, **outs)
    count = 6
    for step in range(5):
        if step == 3:
            new = [2, 0, 1, 1]
            dn.copy_(ints(new))
        graph.replay()
        lens, count, cu, positions, slots, table = os_.extend(new, lens, table, free, count, 6)
        assert dl.tolist() == lens and dc.tolist() == [count] and dt.tolist() == table
        assert outs["positions"].tolist() == positions and outs["slots"].tolist() == slots
        assert outs["cu_tokens"].tolist() == cu
    assert api.device_status() == 0


@pytest.mark.parametrize("lens,done", [
    ([5], [1]), ([5], [0]), ([0, 128, 129], [1, 1, 1]), ([300, -2, 1, 4000], [0, 1, 1, 1]),
    ([70000, 3], [1, 0]), ([i % 500 for i in range(3000)], [i % 3 != 1 for i in range(3000)])])
def test_release(lens, done):
    wide = max(-(-max(n, 0) // PAGE) for n in lens) + 1
    table, free, pages = state(lens, wide, 4, seed=len(lens))
    padded = free + [-9] * (pages - 4)
    args = (ints(done, torch.bool), ints(lens), ints(table), ints(padded), ints([4]))
    after, count = api.nvfp4_kv_release(*args)
    want = os_.release(done, lens, table, padded, 4)
    assert after.tolist() == want[0] and count.tolist() == [want[1]]
    assert args[3].tolist() == want[2] and args[2].tolist() == table
    assert args[1].tolist() == lens and args[4].tolist() == [4]
    assert api.device_status() == 0
    args[3].copy_(ints(padded))
    inplace = api.nvfp4_kv_release(*args, seq_lens_out=args[1], free_count_out=args[4])
    assert inplace[0].tolist() == want[0] and args[4].tolist() == [want[1]]


def test_release_refuses_whole_calls():
    lens = [200, 130, 5]
    table, free, pages = state(lens, 3, 4, seed=1)
    padded = free + [-9] * (pages - 4)

    def call(table=table, lens=lens, free=padded, count=4):
        args = (ints([1, 1, 0], torch.bool), ints(lens), ints(table), ints(free), ints([count]))
        after, n = api.nvfp4_kv_release(*args)
        assert after.tolist() == lens and n.tolist() == [count] and args[3].tolist() == free
        assert api.device_status() == 1

    call(table=[table[0], [table[1][0], pages, -7], table[2]])
    call(table=[[-1] + table[0][1:], table[1], table[2]])
    call(lens=[200, 400, 5])
    call(lens=[200, 2 ** 31 - 1, 5])
    call(free=padded[:7])
    call(count=-1)
    call(count=pages)


@pytest.mark.parametrize("hkv,d", [(3, 128), (8, 64), (1, 128)])
def test_append_by_slots_is_the_append_by_tables(hkv, d):
    g = torch.Generator().manual_seed(d + hkv)
    new, lens = [130, 0, 1, 77], [100, 3, 255, 0]
    table, free, pages = state(lens, 4, 8, seed=4)
    t = sum(new)
    kv = torch.randn(t + 3, 2, hkv, d, generator=g).to(torch.bfloat16).cuda()
    k, v = kv[:, 0], kv[:, 1]  # strided rows, three of them behind the last token
    step, args = run_extend(new, lens, table, free, pages, t + 3)
    a = torch.randint(0, 256, (pages, hkv, 144 * d), dtype=torch.uint8, generator=g).cuda()
    b = a.clone()
    api.nvfp4_kv_append_slots(k, v, step.slots, a)
    api.nvfp4_kv_append(k, v, step.seq_lens, args[2], b, step.cu_tokens)
    assert torch.equal(a, b) and api.device_status() == 0
    none = torch.empty(0, hkv, d, dtype=torch.bfloat16, device="cuda")
    api.nvfp4_kv_append_slots(none, none, step.slots[:0], a)
    assert torch.equal(a, b)


def test_append_by_slots_skips_and_reports_what_is_outside():
    pool = api.nvfp4_kv_pool(2, 1, 64)
    x = torch.ones(5, 1, 64, dtype=torch.bfloat16, device="cuda")
    api.nvfp4_kv_append_slots(x[:2], x[:2], ints([-1, -(1 << 40)], torch.int64), pool)
    assert not bool(pool.any()) and api.device_status() == 0
    api.nvfp4_kv_append_slots(x, x, ints([256, 1 << 40, 255, -1, (1 << 62)], torch.int64), pool)
    assert api.device_status() == 1
    k = pool[1, 0, :64 * 128 // 2].view(128, 32)
    assert not bool(pool[0].any()) and not bool(k[:127].any()) and bool(k[127].all())


def test_no_sequences():
    none, table = ints([]), torch.empty(0, 3, dtype=I32, device="cuda")
    free, count = ints([4, 5, 6]), ints([2])
    step = api.nvfp4_kv_extend(none, none, table, free, count, tokens=4)
    assert step.cu_tokens.tolist() == [0] and step.free_count.tolist() == [2]
    assert step.positions.tolist() == [-1] * 4 and step.slots.tolist() == [-1] * 4
    lens, count = api.nvfp4_kv_release(none.bool(), none, table, free, count)
    assert lens.numel() == 0 and count.tolist() == [2]
