"""Windows and first tokens past 32 bits: as good as all keys, never their low 32 bits."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import _lib, api

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_large_windows_and_sinks():
    g = torch.Generator().manual_seed(1)
    pool = api.nvfp4_kv_pool(3, 1, 64)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(300, 1, 64, generator=g).to(BF16).cuda() for _ in range(2))
    api.nvfp4_kv_append(k, v, lens, table, pool, torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 2, 64, generator=g).to(BF16).cuda()
    want = api.attn_qat_decode(q, pool, table, lens)
    near = api.attn_qat_decode(q, pool, table, lens, window=5)
    assert not torch.equal(near[0], want[0])
    for window, sinks in ((2 ** 32 + 5, 0), (2 ** 31 - 1, 0), (2 ** 31, 0), (2 ** 63, 2 ** 40), (300, 7)):
        got = api.attn_qat_decode(q, pool, table, lens, window=window, sinks=sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # every key is a first one: two ranges of the same keys, in one sum
    got = api.attn_qat_decode(q, pool, table, lens, window=5, sinks=2 ** 32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bad in (dict(window=-1), dict(window=5 - 2 ** 32), dict(window=5, sinks=-2 ** 32)):
        with pytest.raises(_lib.NvqError):
            api.attn_qat_decode(q, pool, table, lens, **bad)
    assert api.device_status() == 0
