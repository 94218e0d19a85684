"""The per-kernel timing files the serving calls under kinds of their own: the training kinds
count what they counted before."""
import ctypes

import pytest
import torch

from nvfp4_fake_quant_gb300 import _lib, api
from nvfp4_fake_quant_gb300 import build as nvbuild

BF16 = torch.bfloat16


def test_kinds_that_can_be_read():
    lib = _lib.load(nvbuild.build())
    n, ms = ctypes.c_int64(-1), ctypes.c_double(-1.0)
    at = ctypes.addressof(n), ctypes.addressof(ms)
    good = set(api.KERNEL_KINDS.values()) | set(api.SERVING_KINDS.values())
    assert len(good) == len(api.KERNEL_KINDS) + len(api.SERVING_KINDS)
    for kind in range(-2, 40):
        assert lib.nvq_timing_read(kind, *at) == (0 if kind in good else 1)


@pytest.mark.gpu
def test_serving_calls_have_their_own_kinds():
    packed = api.NVFP4Linear(128, 256, device="cuda").pack()
    pool = api.nvfp4_kv_pool(1, 1, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    f = api.rope_inv_freq(64, device="cuda")[0]
    api.timing_enable(True)
    try:
        qkv = packed(torch.randn(1, 128, device="cuda").to(BF16)).view(1, 4, 64)
        q, k = api.rope_apply(qkv[:, :2], qkv[:, 2:3], lens - 1, f)
        api.nvfp4_kv_append(k, qkv[:, 3:], lens, table, pool)
        api.attn_qat_decode(q, pool, table, lens)
        got = api.timing_read()
    finally:
        api.timing_enable(False)
    assert {name: n for name, (n, _) in got.items()} == {
        "quantize": 0, "attn_fwd": 0, "bwd_delta": 0, "bwd_dkdv": 0, "bwd_dq": 0, "global_sf": 1,
        "vsa": 0, "linear": 1, "rope": 1, "kv_append": 1, "decode": 1}
    assert all(ms > 0 for n, ms in got.values() if n)
