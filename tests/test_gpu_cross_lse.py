"""lse where every score is exactly 0 (a query of zeros): ln of the number of keys, to fp32's
accuracy, from one key to a long prefix.  With E = 0 the bound of test_gpu_kv_cache.py is
2^-20 + |lse| 2^-23."""
import math

import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from test_gpu_cross import ints, offsets
from test_gpu_kv_cache import BF16, make_pool

pytestmark = pytest.mark.gpu


def check(lse, keys):
    want = torch.tensor([math.log(n) for n in keys], dtype=torch.float64)[:, None]
    err = (lse.cpu().double() - want).abs()
    assert bool((err <= 2.0 ** -20 + want * 2.0 ** -23).all()), float((err * 2.0 ** 20).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [2, 70, 200])
def test_counts_of_keys(d, t):
    """t rows of each of some sequences of every length, and one of 131072 keys (a page again and
    again), which many runs share."""
    h, hkv, wide = 2, 2, 1024
    gen = torch.Generator().manual_seed(d)
    pool = make_pool(1, hkv, d, gen).cuda()
    lens = [*range(1, 40), 100, 127, 128, 129, 200, 255, 257, 383, 511, 700, 1000, 3333, 20000,
            wide * 128]
    b = len(lens)
    table = torch.zeros(b, wide, dtype=torch.int32, device="cuda")
    q = torch.zeros(b * t, h, d, dtype=BF16, device="cuda")
    _, lse = api.attn_qat_cross(q, pool, table, ints(lens), ints(offsets([t] * b)))
    check(lse, [n for n in lens for _ in range(t)])
    _, lse = api.attn_qat_decode_prefix(q[:b], pool, table[:, :1].contiguous(), ints([0] * b), table,
                                        ints(lens))
    check(lse, lens)
    _, lse = api.attn_qat_decode_prefix(q[:b], pool, table[:, :1].contiguous(), ints([77] * b), table,
                                        ints(lens))
    check(lse, [n + 77 for n in lens])
    assert api.device_status() == 0
