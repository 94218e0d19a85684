"""Pins of oracle/serving.py: rotations against complex multiplication and their own
inverse, cache records against the pinned quantizer, single-token attention against the
last row of the causal attention oracle, the visible-key rule by hand."""
import torch

from nvfp4_fake_quant_gb300 import api, workloads
from oracle import attention as oa
from oracle import serving as os_
from oracle.nvfp4 import fq

F64 = torch.float64


def test_rope_is_a_complex_rotation_and_its_inverse_undoes_it():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 3, 64, generator=g, dtype=F64)
    pos = torch.tensor([0, 1, 7, -3, 100000])
    f, _ = api.rope_inv_freq(32)
    y = os_.rope(x, pos, f, interleaved=True)
    z = torch.view_as_complex(x[..., :32].reshape(5, 3, 16, 2).contiguous())
    turn = torch.polar(torch.ones(5, 16, dtype=F64), pos[:, None].to(F64) * f)
    want = torch.view_as_real(z * turn[:, None]).flatten(-2)
    assert torch.allclose(y[..., :32], want, atol=1e-12) and torch.equal(y[..., 32:], x[..., 32:])
    assert torch.equal(y[0], x[0])
    for inter in (False, True):
        y = os_.rope(x, pos, f, inter, mscale=2.0)
        assert torch.allclose(os_.rope(y, pos, f, inter, mscale=0.5, inverse=True), x, atol=1e-12)


def test_rope_axes_use_their_own_positions():
    x = torch.randn(4, 1, 32, generator=torch.Generator().manual_seed(2), dtype=F64)
    f = torch.rand(16, generator=torch.Generator().manual_seed(3), dtype=F64)
    pos = torch.tensor([[1, 2, 3], [0, 0, 0], [5, 0, 9], [2, 2, 2]])
    y = os_.rope(x, pos, f, axis_pairs=(4, 6, 6))
    for lo, hi, a in ((0, 4, 0), (4, 10, 1), (10, 16, 2)):
        one = os_.rope(x, pos[:, a], f)
        assert torch.equal(y[..., lo:hi], one[..., lo:hi])
        assert torch.equal(y[..., 16 + lo:16 + hi], one[..., 16 + lo:16 + hi])


def test_inv_freq_scalings():
    f0, m0 = api.rope_inv_freq(128)
    assert f0[0] == 1.0 and m0 == 1.0 and abs(f0[32] - 0.01) < 1e-15
    f, m = api.rope_inv_freq(128, scaling="linear", factor=4.0)
    assert torch.equal(f, f0 / 4) and m == 1.0
    f, m = api.rope_inv_freq(128, scaling="theta", factor=4.0)
    assert f[0] == 1.0 and abs(f[-1] / (f0[-1] / 4) - 1) < 1e-12
    f, m = api.rope_inv_freq(128, scaling="by_parts", factor=4.0, original_len=8192)
    turns = 8192 * f0 / (2 * torch.pi)
    assert torch.equal(f[turns > 32], f0[turns > 32])
    assert torch.allclose(f[turns < 1], f0[turns < 1] / 4, rtol=1e-15) and m > 1.0
    assert bool((f <= f0).all() and (f >= f0 / 4 * (1 - 1e-15)).all())


def test_records_round_trip_the_quantizer():
    x = workloads.random_matrix(24, 128, seed=5).to(F64)
    codes, scales = os_.pack(x)
    assert torch.equal(os_.unpack(codes, scales), fq(x))


def test_visible_rule():
    assert os_.visible(5, 0, 3) == [0, 1, 2, 3, 4]
    assert os_.visible(5, 2, 0) == [3, 4]
    assert os_.visible(5, 2, 1) == [0, 3, 4]
    assert os_.visible(5, 9, 1) == [0, 1, 2, 3, 4]
    assert os_.visible(0, 2, 1) == []


def test_decode_is_the_last_row_of_the_causal_oracle():
    n, h, d = 150, 2, 64
    inp = workloads.attn_inputs(1, n, n, h, d, seed=6, causal=True)
    pool = torch.zeros(4, h, 144 * d, dtype=torch.uint8)
    table = torch.tensor([[2, 0]])
    for x, at_c, at_s in ((inp.k, 0, 128 * d), (inp.v, 64 * d, 136 * d)):
        codes, scales = os_.pack(x[0].to(F64))
        for j in range(n):
            p, r = int(table[0, j // 128]), j % 128
            pool[p, :, at_c + r * d // 2:at_c + (r + 1) * d // 2] = codes[j]
            pool[p, :, at_s + r * d // 16:at_s + (r + 1) * d // 16] = scales[j]
    o, lse, mag, err = os_.decode(inp.q[:, -1].to(F64), pool, table, [n], inp.scale)
    want = oa.attn_fwd_hp(inp.q, inp.k, inp.v, inp.scale, True)[:, -1]
    _, lse_ref, _ = oa.attn_fwd(inp.q, inp.k, inp.v, inp.scale, True)
    assert torch.allclose(o, want, atol=1e-12)
    assert torch.allclose(lse[0], lse_ref[0, :, -1], atol=1e-12)
    assert bool((mag >= o.abs() - 1e-12).all()) and bool((err > 0).all())
