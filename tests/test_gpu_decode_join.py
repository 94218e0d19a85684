"""Decode of few sequences with many query heads on one KV head, long enough that the parts
of a segment are joined by blocks of 1024 threads, sixteen heads a run (over 64 runs a
segment: one to four segments of some 150 pages and more).  Bounds of test_gpu_kv_cache.py.
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_kv_cache import PAGE, check_decode, make_pool, spoil

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("h,hkv,d,lens,window,sinks", [
    (16, 1, 64, [20011], 0, 0), (16, 1, 128, [19999], 0, 0), (12, 1, 128, [20480, 130], 0, 0),
    (40, 1, 64, [19600], 0, 0), (9, 1, 128, [19500, 0, 3], 0, 0), (32, 2, 128, [19457], 0, 0),
    (16, 1, 128, [25000], 20000, 5), (24, 2, 64, [21000], 300, 130)])
def test_many_parts_of_sixteen_heads(h, hkv, d, lens, window, sinks):
    g = torch.Generator().manual_seed(h + d + lens[0])
    pages, width = 48, -(-max(lens) // PAGE) + 1
    pool = make_pool(pages, hkv, d, g)  # pages reused, the last ones spoilt behind the tokens
    vmax = float(os_.unpack(*os_.record_parts(pool, d)[1::2]).abs().max())
    table = torch.randint(0, pages - len(lens), (len(lens), width), generator=g, dtype=torch.int32)
    for i, n in enumerate(lens):
        table[i, max(0, (n - 1) // PAGE)] = pages - 1 - i
    spoil(pool, table, lens, d)
    b = len(lens)
    q = torch.randn(b, h, d, generator=g).to(BF16)
    ref = os_.decode(q, pool, table, lens, d ** -0.5, window, sinks)
    ws = torch.full((api.attn_qat_decode_workspace(b, h, hkv, d, width),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    args = (q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            d ** -0.5, window, sinks)
    o, lse = api.attn_qat_decode(*args, workspace=ws)
    assert api.device_status() == 0
    check_decode(o, lse, ref, max(lens), vmax)
    o2, lse2 = api.attn_qat_decode(*args, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
