"""The serving calls tell autograd what they overwrite: a graph that saved an output tensor
refuses its backward instead of taking the new values."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def saved(t):
    """A result whose backward needs t's values."""
    leaf = torch.ones((), device=t.device, requires_grad=True)
    return (leaf.to(t.dtype) * t).sum()


def test_rotation_in_place():
    q, k = (torch.randn(5, 2, 64, device="cuda").to(BF16) for _ in range(2))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    f = api.rope_inv_freq(64, device="cuda")[0]
    before = saved(q), saved(k)
    api.rope_apply(q, k, pos, f)  # outputs of its own: nothing is lost
    saved(q).backward()
    api.rope_apply(q, k, pos, f, q_out=q, k_out=k)
    for y in before:
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    saved(q).backward()


def test_given_outputs():
    w = torch.randn(32, 128, device="cuda").to(BF16)
    codes, scales = api.nvfp4_quantize_tiled(w)
    x = torch.randn(2, 128, device="cuda").to(BF16)
    out = torch.zeros(2, 32, dtype=BF16, device="cuda")
    before = saved(out)
    api.nvfp4_linear_packed_fwd(x, codes, scales, out=out)
    with pytest.raises(RuntimeError, match="inplace"):
        before.backward()

    pool = api.nvfp4_kv_pool(1, 2, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    kv = torch.randn(1, 2, 64, device="cuda").to(BF16)
    version = pool._version
    api.nvfp4_kv_append(kv, kv, lens, table, pool)
    assert pool._version > version
    o, lse = torch.zeros(1, 4, 64, dtype=BF16, device="cuda"), torch.zeros(1, 4, device="cuda")
    before = saved(o), saved(lse)
    api.attn_qat_decode(kv.repeat(1, 2, 1), pool, table, lens, o=o, lse=lse)
    for y in before:
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    assert api.device_status() == 0


def test_inference_tensors():
    with torch.inference_mode():
        q = torch.randn(5, 2, 64, device="cuda").to(BF16)
        pos = torch.arange(5, dtype=torch.int32, device="cuda")
        f = api.rope_inv_freq(64, device="cuda")[0]
        want = api.rope_apply(q, None, pos, f)[0]
        api.rope_apply(q, None, pos, f, q_out=q)
        assert torch.equal(q, want)
