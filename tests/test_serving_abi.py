"""Refusals of the single-token serving calls and the rotary positions: wrong sizes,
strides, pointers and workspaces return their status on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from nvfp4_fake_quant_gb300 import _lib, api
from nvfp4_fake_quant_gb300 import build as nvbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x100000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load(nvbuild.build())


def test_rope_refusals(lib):
    def rope(q=A, ld_q=256, qo=A + 65536, ld_qo=256, hq=2, k=A, ld_k=128, ko=A + 65536, ld_ko=128,
             hk=1, t=4, d=128, rot=128, inter=0, pos=A, axes=1, pairs=(64,), freq=A, ms=1.0, inv=0):
        ap = None if pairs is None else (ctypes.c_int * max(1, len(pairs)))(*pairs)
        return lib.rope_apply(q, ld_q, qo, ld_qo, hq, k, ld_k, ko, ld_ko, hk, t, d, rot, inter, pos,
                              axes, ap, freq, ms, inv, None)
    assert rope(t=0, q=None, pos=None) == OK  # nothing to do, nothing touched
    for bad in (dict(t=-1), dict(hq=0), dict(hk=-1), dict(q=None), dict(q=A + 8), dict(qo=None),
                dict(ld_q=248), dict(ld_q=260), dict(ld_qo=255), dict(k=None), dict(ko=A + 4),
                dict(ld_k=120), dict(ld_ko=100), dict(pos=None), dict(pos=A + 2), dict(freq=None),
                dict(freq=A + 4), dict(ms=0.0), dict(ms=float("nan")), dict(ms=float("inf")),
                dict(inter=2), dict(inv=-1), dict(axes=0), dict(axes=4), dict(pairs=None),
                dict(pairs=(63,)), dict(pairs=(-1, 65), axes=2), dict(rot=144), dict(rot=0),
                dict(qo=A, ld_qo=264)):
        assert rope(**bad) == INVALID, bad
    for bad in (dict(rot=24, pairs=(12,)), dict(d=72, rot=64, pairs=(32,)),
                dict(d=272, rot=64, pairs=(32,), ld_q=1024, ld_k=1024, ld_qo=1024, ld_ko=1024)):
        assert rope(**bad) == UNSUPPORTED, bad


def test_append_refusals(lib):
    def app(k=A, ld_k=256, v=A, ld_v=256, t=3, b=3, hkv=2, d=128, cu=None, lens=A, table=A,
            ld_t=4, mp=4, pool=A, pages=8):
        return lib.nvfp4_kv_append(k, ld_k, v, ld_v, t, b, hkv, d, cu, lens, table, ld_t, mp, pool,
                                   pages, None)
    assert app(t=0, k=None, pool=None) == OK
    for bad in (dict(t=-1), dict(b=0), dict(hkv=0), dict(t=4), dict(k=None), dict(v=A + 8),
                dict(ld_k=248), dict(ld_v=260), dict(cu=A + 1), dict(lens=None), dict(lens=A + 2),
                dict(table=None), dict(ld_t=3), dict(mp=0), dict(mp=1 << 25), dict(pool=None),
                dict(pool=A + 8), dict(pages=0), dict(pages=1 << 31)):
        assert app(**bad) == INVALID, bad
    assert app(d=96) == UNSUPPORTED
    assert lib.nvfp4_kv_page_bytes(8, 128) == 8 * 18432
    assert lib.nvfp4_kv_page_bytes(1, 64) == 9216
    assert lib.nvfp4_kv_page_bytes(0, 64) == 0 and lib.nvfp4_kv_page_bytes(2, 96) == 0


def test_decode_refusals(lib):
    def dec(q=A, ld_q=1024, pool=A, pages=8, table=A, ld_t=4, mp=4, lens=A, b=2, h=8, hkv=2, d=128,
            scale=0.1, window=0, sinks=0, o=A, lse=None, ws=A, ws_bytes=BIG):
        return lib.attn_qat_decode(q, ld_q, pool, pages, table, ld_t, mp, lens, b, h, hkv, d, scale,
                                   window, sinks, o, lse, ws, ws_bytes, None)
    for bad in (dict(b=0), dict(h=0), dict(hkv=0), dict(hkv=3), dict(mp=0), dict(ld_t=2),
                dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1),
                dict(q=None), dict(q=A + 8), dict(ld_q=1016), dict(ld_q=1028), dict(pool=None),
                dict(pool=A + 4), dict(pages=0), dict(table=None), dict(lens=None),
                dict(lens=A + 2), dict(o=None), dict(o=A + 8), dict(lse=A + 2)):
        assert dec(**bad) == INVALID, bad
    assert dec(d=96) == UNSUPPORTED and dec(b=70000) == UNSUPPORTED
    assert dec(ws=None) == WORKSPACE and dec(ws=A + 16) == WORKSPACE and dec(ws_bytes=0) == WORKSPACE
    assert lib.attn_qat_decode_workspace(2, 8, 2, 128, 4) > 0
    assert lib.attn_qat_decode_workspace(2, 8, 3, 128, 4) == 0
    assert lib.attn_qat_decode_workspace(2, 8, 2, 80, 4) == 0


def test_decode_refuses_an_output_over_its_queries(lib):
    def dec(q, o, ld_q=1024):
        return lib.attn_qat_decode(q, ld_q, A, 8, A, 4, 4, A, 2, 8, 2, 128, 0.1, 0, 0, o, None, A,
                                   BIG, None)
    rows = 2 * 8 * 128 * 2  # bytes of q and of o
    assert dec(A, A) == INVALID
    assert dec(A, A + rows - 16) == INVALID and dec(A + rows - 16, A) == INVALID
    assert dec(A, A + rows, ld_q=2048) == INVALID  # inside a strided q


def test_decode_refuses_more_tiles_than_its_cut_takes(lib):
    assert lib.attn_qat_decode_workspace(65535, 32767, 32767, 64, (1 << 22) + 300) == 0
    assert lib.attn_qat_decode_workspace(65535, 32767, 32767, 64, 1 << 20) > 0


def test_packed_linear_refusals(lib):
    def lin(x=A, ld=128, c=A, s=A, wg=None, bias=None, m=2, n=32, k=128, xg=None, out=A, ws=A,
            ws_bytes=BIG):
        return lib.nvfp4_linear_packed_fwd(x, ld, c, s, wg, bias, m, n, k, xg, out, ws, ws_bytes,
                                           None)
    for bad in (dict(m=0), dict(n=0), dict(k=0), dict(x=None), dict(x=A + 2), dict(ld=64),
                dict(ld=132), dict(c=None), dict(s=A + 8), dict(bias=A + 2), dict(out=None),
                dict(wg=A + 1), dict(xg=A + 2)):
        assert lin(**bad) == INVALID, bad
    assert lin(k=96) == UNSUPPORTED and lin(n=24) == UNSUPPORTED
    assert lin(ws=None) == WORKSPACE and lin(ws=A + 64) == WORKSPACE
    need = lib.nvfp4_linear_packed_workspace(2, 32, 128)
    assert need > 0 and lin(ws_bytes=need - 1) == WORKSPACE
    assert lib.nvfp4_linear_packed_workspace(2, 24, 128) == 0


def test_packed_linear_leaves_x_past_31_bits_of_blocks_to_the_gemm(lib):
    # 64 x 2^30 elements: 2^32 blocks, over the few-rows kernel's 32-bit index.  The GEMM's
    # workspace holds x's codes and the scales of whole tiles of 128 rows
    k = 1 << 30
    assert lib.nvfp4_linear_packed_workspace(64, 16, k) >= 64 * k // 2 + 128 * k // 16
    # 31 rows stay below: scales of 1 KB per 256 elements
    assert lib.nvfp4_linear_packed_workspace(31, 16, k) == 31 * k // 2 + k // 256 * 1024 + 256


def test_python_layer_refuses_host_tensors_and_bad_shapes():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pos, f = torch.zeros(2, dtype=torch.int32), api.rope_inv_freq(64)[0]
    with pytest.raises(ValueError, match="CUDA"):
        api.rope_apply(q, None, pos, f)
    with pytest.raises(ValueError, match="CUDA"):
        api.nvfp4_linear_packed_fwd(q[0], torch.zeros(16, 32, dtype=torch.uint8), q)
    with pytest.raises(ValueError, match="CUDA"):
        api.nvfp4_kv_append(q, q, pos, pos, pos)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_qat_decode(q, pos, pos, pos)
    with pytest.raises(ValueError):
        api.rope_inv_freq(63)
    with pytest.raises(ValueError):
        api.rope_inv_freq(64, scaling="other")
    with pytest.raises(ValueError):
        api.Rotary(64, inv_freq=f[:-1])
    with pytest.raises(ValueError):
        api.nvfp4_kv_pool(2, 2, 96, device="cpu")
    assert api.nvfp4_kv_pool(2, 3, 64, device="cpu").shape == (2, 3, 9216)


def test_rotary_keeps_its_frequencies_when_the_model_changes_type():
    rot = api.Rotary(64)
    f = rot.inv_freq.clone()
    holder = torch.nn.Sequential(torch.nn.Linear(2, 2), rot)
    for change in (lambda m: m.to(torch.bfloat16), lambda m: m.half(), lambda m: m.float()):
        change(holder)
        assert rot.inv_freq.dtype == torch.float64 and torch.equal(rot.inv_freq, f)
    assert holder[0].weight.dtype == torch.float32
