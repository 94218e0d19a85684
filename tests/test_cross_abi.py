"""Refusals of the attention of many rows over the cache and of the decode behind a prefix: wrong
sizes, strides, pointers and workspaces return their status on the host, before any CUDA call."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import _lib, api
from nvfp4_fake_quant_gb300 import build as nvbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x100000
O = 1 << 32  # outputs, far from the queries
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load(nvbuild.build())


def test_cross_refusals(lib):
    def cross(q=A, ld_q=1024, t=6, pool=A, pages=8, table=A, ld=4, mp=4, lens=A, cu=None, b=2, h=8,
              hkv=2, d=128, scale=0.1, o=O, lse=None, ws=A, n=BIG):
        return lib.attn_qat_cross(q, ld_q, t, pool, pages, table, ld, mp, lens, cu, b, h, hkv, d,
                                  scale, o, lse, ws, n, None)
    for bad in (dict(t=0), dict(t=-1), dict(b=0), dict(h=0), dict(hkv=0), dict(hkv=3), dict(mp=0),
                dict(mp=1 << 25), dict(ld=3), dict(scale=0.0), dict(scale=float("inf")), dict(t=7),
                dict(cu=A + 2), dict(q=None), dict(q=A + 8), dict(ld_q=1016), dict(ld_q=1028),
                dict(pool=None), dict(pool=A + 8), dict(pages=0), dict(table=None), dict(lens=None),
                dict(lens=A + 2), dict(o=None), dict(o=O + 8), dict(lse=A + 2), dict(o=A),
                dict(o=A + 6 * 2048 - 16), dict(q=O + 6 * 2048 - 16)):
        assert cross(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(b=65536, t=65536), dict(t=(1 << 31) // 8, cu=A),
                dict(b=65535, t=65535, cu=A, h=256, hkv=256, ld_q=1 << 16, mp=1 << 20, ld=1 << 20),
                dict(pages=1 << 30)):
        assert cross(**bad) == UNSUPPORTED, bad
    assert cross(ws=None) == WORKSPACE and cross(ws=A + 16) == WORKSPACE
    need = lib.attn_qat_cross_workspace(6, 2, 8, 2, 128, 4)
    assert need > 0 and cross(n=need - 1) == WORKSPACE
    assert lib.attn_qat_cross_workspace(6, 2, 8, 3, 128, 4) == 0
    assert lib.attn_qat_cross_workspace(6, 2, 8, 2, 80, 4) == 0
    # one token a sequence may take the single-token call
    assert lib.attn_qat_cross_workspace(64, 64, 16, 16, 64, 12) >= \
        lib.attn_qat_decode_workspace(64, 16, 16, 64, 12)


def test_prefix_refusals(lib):
    def dec(q=A, ld_q=1024, pool=A, pages=8, table=A, ld=4, mp=4, lens=A, ptable=A, ld_p=3, pp=3,
            plens=A, cu=None, s=2, b=4, h=8, hkv=2, d=128, scale=0.1, o=O, lse=None, ws=A, n=BIG):
        return lib.attn_qat_decode_prefix(q, ld_q, pool, pages, table, ld, mp, lens, ptable, ld_p,
                                          pp, plens, cu, s, b, h, hkv, d, scale, o, lse, ws, n,
                                          None)
    for bad in (dict(b=0), dict(s=0), dict(s=3), dict(h=0), dict(hkv=3), dict(mp=0), dict(pp=0),
                dict(pp=1 << 25), dict(ld=3), dict(ld_p=2), dict(scale=-1.0),
                dict(scale=float("nan")), dict(cu=A + 1), dict(q=None), dict(q=A + 2),
                dict(ld_q=1020), dict(pool=None), dict(pages=0), dict(table=None),
                dict(lens=None), dict(ptable=None), dict(ptable=A + 2), dict(plens=None),
                dict(plens=A + 2), dict(o=None), dict(o=A), dict(o=A + 4 * 2048 - 16),
                dict(lse=A + 1)):
        assert dec(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(b=70000), dict(s=65536, cu=A), dict(pages=1 << 30)):
        assert dec(**bad) == UNSUPPORTED, bad
    assert dec(ws=None) == WORKSPACE and dec(ws=A + 128) == WORKSPACE
    need = lib.attn_qat_decode_prefix_workspace(4, 2, 8, 2, 128, 4, 3)
    assert need > lib.attn_qat_decode_workspace(4, 8, 2, 128, 4) and dec(n=need - 1) == WORKSPACE
    assert lib.attn_qat_decode_prefix_workspace(4, 2, 8, 3, 128, 4, 3) == 0
    assert lib.attn_qat_decode_prefix_workspace(4, 0, 8, 2, 128, 4, 3) == 0


def test_python_layer_refusals():
    n, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool = api.nvfp4_kv_pool(1, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_qat_cross(q, pool, table, n)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_qat_decode_prefix(q[:2], pool, table, n, table, n)
