"""lse of rows that see a NaN among their keys: -inf from every call and in every form of it, as
attn_qat_decode gives it (their o is NaN)."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from test_gpu_cross import ints
from test_gpu_kv_cache import BF16, make_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("own", [0, 1, 5, 300])
def test_lse(d, own):
    h, hkv, b = 4, 2, 5
    g = torch.Generator().manual_seed(own + d)
    pool = make_pool(8, hkv, d, g)
    pool[1, 1, 128 * d + 7 * d // 16] = 0x7F  # K's scales, page 1, head 1, key 7
    pool = pool.cuda()
    q = torch.randn(b, h, d, generator=g).to(BF16).cuda()
    clean, spoilt = ints([2, 3]), ints([0, 1])
    mine, lens = ints([[4, 5, 6]] * b), ints([own] * b)
    sees = torch.zeros(b, h, dtype=torch.bool, device="cuda")

    def check(o, lse):
        assert torch.equal(o.isnan().any(-1), sees) and torch.equal(o.isnan().all(-1), sees)
        assert torch.equal(lse == -float("inf"), sees) and bool(torch.isfinite(lse[~sees]).all())

    # among a prefix's keys
    sees[:3, 2:] = True
    check(*api.attn_qat_decode_prefix(q, pool, mine, lens, torch.stack((spoilt, clean)),
                                      ints([200, 200]), ints([0, 3, 5])))
    # among an encoder's
    check(*api.attn_qat_cross(q, pool, torch.stack((spoilt, clean)), ints([200, 200]),
                              ints([0, 3, 5])))
    # among the own keys
    sees[:] = False
    sees[1, 2:] = True
    mine = clean.expand(b, 2).clone()
    mine[1] = spoilt
    check(*api.attn_qat_decode(q, pool, mine, ints([200] * b)))
    check(*api.attn_qat_cross(q, pool, mine, ints([200] * b)))
    if own:
        check(*api.attn_qat_decode_prefix(q, pool, mine, ints([200] * b), clean[None],
                                          ints([min(own, 256)])))
    assert api.device_status() == 0
