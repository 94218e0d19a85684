"""A step without sequences goes through every serving call: nothing is launched, the outputs
are empty; wrong sizes are refused all the same."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import _lib, api

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_a_step_of_no_sequences():
    h, hkv, d, hidden = 4, 2, 64, 128
    packed = api.NVFP4Linear(hidden, (h + 2 * hkv) * d, device="cuda").pack()
    back = api.NVFP4Linear(h * d, hidden, device="cuda").pack()
    rot = api.Rotary(d, device="cuda")
    pool = api.nvfp4_kv_pool(2, hkv, d)
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    qkv = packed(torch.empty(0, hidden, dtype=BF16, device="cuda")).view(0, h + 2 * hkv, d)
    q, k = rot(qkv[:, :h], qkv[:, h:h + hkv], none)
    api.nvfp4_kv_append(k, qkv[:, h + hkv:], none, table, pool)
    api.nvfp4_kv_append(k, qkv[:, h + hkv:], none, table, pool,
                        torch.zeros(1, dtype=torch.int32, device="cuda"))
    o, lse = api.attn_qat_decode(q, pool, table, none)
    assert o.shape == (0, h, d) and o.dtype == BF16
    assert lse.shape == (0, h) and lse.dtype == torch.float32
    assert back(o.reshape(0, h * d)).shape == (0, hidden)
    assert back(o.new_empty(3, 0, h * d)).shape == (3, 0, hidden)
    assert not bool(pool.any()) and api.device_status() == 0


def test_wrong_sizes_are_refused_without_sequences():
    pool = torch.zeros(2, 2, 144 * 64, dtype=torch.uint8, device="cuda")
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    with pytest.raises(_lib.NvqError):  # 3 heads over 2
        api.attn_qat_decode(torch.empty(0, 3, 64, dtype=BF16, device="cuda"), pool, table, none)
    with pytest.raises(ValueError):  # tokens of no sequence
        api.nvfp4_kv_append(*[torch.zeros(1, 2, 64, dtype=BF16, device="cuda")] * 2, none, table, pool)
    odd = torch.zeros(2, 2, 144 * 96, dtype=torch.uint8, device="cuda")
    x = torch.empty(0, 2, 96, dtype=BF16, device="cuda")
    with pytest.raises(_lib.NvqError):  # heads of 96
        api.nvfp4_kv_append(x, x, none, table, odd)
    codes, scales = api.nvfp4_quantize_tiled(torch.zeros(24, 128, dtype=BF16, device="cuda"))
    with pytest.raises(_lib.NvqError):  # 24 rows of weights
        api.nvfp4_linear_packed_fwd(torch.empty(0, 128, dtype=BF16, device="cuda"), codes, scales)
