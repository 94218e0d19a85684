"""A workspace that is a broadcast or strided view has fewer bytes than its shape says, or
others' between its own: refused on the host."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def views():
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    return buf, (buf[:1].expand(1 << 24), buf[::2], buf.view(256, 256).t())


def test_packed_linear():
    codes, scales = api.nvfp4_quantize_tiled(torch.zeros(32, 128, dtype=BF16, device="cuda"))
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    buf, bad = views()
    for ws in bad:
        with pytest.raises(ValueError, match="workspace"):
            api.nvfp4_linear_packed_fwd(x, codes, scales, workspace=ws)
    assert not bool(buf.any())
    api.nvfp4_linear_packed_fwd(x, codes, scales, workspace=buf)


def test_decode():
    pool = api.nvfp4_kv_pool(1, 2, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    buf, bad = views()
    for ws in bad:
        with pytest.raises(ValueError, match="workspace"):
            api.attn_qat_decode(q, pool, table, lens, workspace=ws)
    assert not bool(buf.any())
    api.attn_qat_decode(q, pool, table, lens, workspace=buf)
