"""One token a sequence with many query heads on a KV head: the single-token kernel up to 16, the
many rows' from 17 on; the values of both, with and without offsets."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from test_gpu_cross import ints, offsets, queries, reference, vmax_of
from test_gpu_kv_cache import check_decode, make_pool, spoil, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,hkv", [(15, 1), (32, 2), (17, 1), (34, 2), (64, 2), (130, 1), (256, 1),
                                   (257, 1)])
def test_values_and_kernel(h, hkv, d):
    lens = [300, 0, 1, 128, 641]
    b = len(lens)
    g = torch.Generator().manual_seed(h + d)
    table, pages = tables(lens, 6, g)
    pool = make_pool(pages, hkv, d, g)
    vmax = vmax_of(pool, d)
    spoil(pool, table, lens, d)
    q = queries(b, h, d, g)
    ref = reference(q, pool, table, lens, offsets([1] * b), d ** -0.5)
    args = (q.cuda(), pool.cuda(), table.cuda(), ints(lens))
    api.timing_enable(True)
    try:
        got = api.attn_qat_cross(*args)
        kinds = {k for k, (n, _) in api.timing_read().items() if n}
    finally:
        api.timing_enable(False)
    assert kinds == {"decode" if h // hkv <= 16 else "cross"}
    check_decode(*got, ref, max(lens), vmax)
    with_offsets = api.attn_qat_cross(*args, ints(offsets([1] * b)))
    check_decode(*with_offsets, ref, max(lens), vmax)
    if h // hkv > 16:
        assert torch.equal(got[0], with_offsets[0]) and torch.equal(got[1], with_offsets[1])
    assert api.device_status() == 0


def test_workspace_is_enough_for_either():
    for h in (8, 16, 17, 256):
        for b in (1, 64, 1000):
            n = api.attn_qat_cross_workspace(b, b, h, 1, 64, 40)
            assert n >= api.attn_qat_decode_workspace(b, h, 1, 64, 40)
