"""Second derivatives through api.Rotary.  On the CPU the kernel is replaced by the oracle's
rotation in float64, so that the autograd function alone is checked, by torch's numerical
derivatives; on the GPU the kernel's own values are used."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_

F64, BF16 = torch.float64, torch.bfloat16


def oracle_rope(q, k, positions, inv_freq, interleaved=False, axis_pairs=None, mscale=1.0,
                inverse=False):
    """Like the kernel's call, unknown to autograd."""
    return tuple(os_.rope(x.detach(), positions, inv_freq, interleaved, axis_pairs, mscale, inverse)
                 for x in (q, k))


@pytest.mark.parametrize("interleaved,pairs", [(False, None), (True, (3, 5))])
def test_numerical_derivatives(interleaved, pairs, monkeypatch):
    monkeypatch.setattr(api, "rope_apply", oracle_rope)
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(2, 3, h, 20, generator=g, dtype=F64, requires_grad=True) for h in (2, 1))
    axes = 1 if pairs is None else len(pairs)
    pos = torch.randint(0, 50, (3, axes), generator=g, dtype=torch.int32)
    rot = api.Rotary(16, interleaved, pairs, scaling="by_parts", factor=4.0)
    assert torch.autograd.gradcheck(lambda *x: rot(*x, pos), (q, k))
    assert torch.autograd.gradgradcheck(lambda *x: rot(*x, pos), (q, k))
    # one of the two inputs alone
    assert torch.autograd.gradgradcheck(lambda x: rot(x, k.detach(), pos)[0], (q,))


def test_a_penalty_on_the_gradient_reaches_the_input(monkeypatch):
    """q enters the loss by the rotation and beside it: with (J q)^4 / 12, the derivative is
    g = J^T (J q)^3 / 3, that of <g, u> is J^T ((J q)^2 J u)."""
    monkeypatch.setattr(api, "rope_apply", oracle_rope)
    gen = torch.Generator().manual_seed(2)
    q, k, u = (torch.randn(4, 2, 16, generator=gen, dtype=F64) for _ in range(3))
    q.requires_grad_()
    pos = torch.arange(4, dtype=torch.int32)
    rot = api.Rotary(16)
    y = rot(q, k, pos)[0]
    g, = torch.autograd.grad((y ** 4).sum() / 12 + (q ** 2).sum() / 2, q, create_graph=True)
    gg, = torch.autograd.grad((g * u).sum(), q)
    with torch.no_grad():
        ju = os_.rope(u, pos, rot.inv_freq)
        want = os_.rope(y ** 2 * ju, pos, rot.inv_freq, inverse=True) + u
    assert torch.allclose(gg, want, rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
def test_second_derivative_on_the_device():
    """The double backward's rotation is the forward's: equal bit for bit."""
    gen = torch.Generator().manual_seed(3)
    q, k, gy, u = (torch.randn(2, 9, 3, 64, generator=gen).to(BF16).cuda() for _ in range(4))
    gy.requires_grad_()
    q.requires_grad_()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    rot = api.Rotary(32, interleaved=True, device="cuda", scaling="by_parts", factor=4.0)
    y = rot(q, k, pos)[0]
    g, = torch.autograd.grad(y, q, gy, create_graph=True)
    got, = torch.autograd.grad(g, gy, u)
    want = rot(u, k, pos)[0]
    assert torch.equal(got, want) and api.device_status() == 0
