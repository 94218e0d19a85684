"""Rotary positions on the GPU against float64 (oracle/serving.py).

Bound per element: half a bf16 step of the result (2^-8 relative) plus the fp32 angle, sine
and products: the fraction of a turn is rounded to fp32 (2^-26 turns = 2^-23 rad), sine and
cosine add 2 ulp (2^-23) and the two products and their sum three half-steps (2^-23 in
all), in units of mscale (|x1| + |x2|): 2^-21 of it.
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def bound(x, ref, rot, interleaved, mscale):
    i = torch.arange(rot // 2)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a = x.double().abs()
    s = torch.zeros_like(a)
    s[..., one] = s[..., two] = a[..., one] + a[..., two]
    return ref.abs() * 2.0 ** -8 + s * mscale * 2.0 ** -21


CASES = [  # t, hq, hk, d, rot, interleaved, axis_pairs, far
    (1, 1, 0, 64, 64, False, None, 1), (1, 12, 12, 128, 128, True, None, 1 << 20),
    (7, 3, 1, 128, 64, False, None, 1 << 31), (130, 5, 2, 64, 48, True, None, 4096),
    (33, 2, 2, 16, 16, False, None, 100), (5, 1, 1, 256, 256, True, (42, 43, 43), 500),
    (2500, 2, 1, 128, 96, False, (16, 0, 32), 60), (20000, 1, 1, 64, 64, True, (10, 22), 60),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:6])))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_parity(case, inverse):
    t, hq, hk, d, rot, inter, pairs, far = case
    g = torch.Generator().manual_seed(t + d)
    # rows of a wider buffer, with guard columns that must stay as they are
    buf = torch.randn(t, (hq + hk) * d + 24, generator=g).to(BF16).cuda()
    q, k = buf[:, 8:8 + hq * d].view(t, hq, d), buf[:, 16 + hq * d:16 + (hq + hk) * d]
    k = k.view(t, hk, d) if hk else None
    axes = 1 if pairs is None else len(pairs)
    pos = torch.randint(-far if far > 1 else 0, far, (t, axes), generator=g).int()
    f, ms = api.rope_inv_freq(rot, scaling="by_parts", factor=8.0)
    qo, ko = api.rope_apply(q, k, pos.cuda(), f.cuda(), inter, pairs, ms, inverse)
    assert (ko is None) == (hk == 0) and api.device_status() == 0
    refs = []
    for x, y in ((q, qo), (k, ko)):
        if x is None:
            continue
        ref = os_.rope(x.cpu(), pos, f, inter, pairs, ms, inverse)
        refs.append(ref)
        err = (y.cpu().double() - ref).abs()
        assert bool((err <= bound(x.cpu(), ref, rot, inter, ms)).all()), float(err.max())
        assert torch.equal(y[..., rot:], x[..., rot:])
    # in place, on the strided rows: the same values, the columns around them untouched
    before = buf.clone()
    api.rope_apply(q, k, pos.cuda(), f.cuda(), inter, pairs, ms, inverse, q_out=q, k_out=k)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    edges = [slice(0, 8), slice(8 + hq * d, 16 + hq * d), slice(16 + (hq + hk) * d, None)]
    assert all(torch.equal(buf[:, e], before[:, e]) for e in edges)


def test_no_tokens():
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    qo, ko = api.rope_apply(q, q, torch.empty(0, dtype=torch.int32, device="cuda"),
                            api.rope_inv_freq(64, device="cuda")[0])
    assert qo.shape == ko.shape == (0, 2, 64)


def test_gradients_are_the_formula_s_and_differences():
    g = torch.Generator().manual_seed(9)
    t, d = 40, 64
    q, k, gq, gk = (torch.randn(t, 2, d, generator=g).to(BF16).cuda() for _ in range(4))
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    rot = api.Rotary(32, interleaved=True, device="cuda", scaling="by_parts", factor=4.0)
    qr, kr = q.clone().requires_grad_(), k.clone().requires_grad_()
    qo, ko = rot(qr, kr, pos)
    torch.autograd.backward((qo, ko), (gq, gk))
    f = rot.inv_freq.cpu()
    for x, gy, got in ((q, gq, qr.grad), (k, gk, kr.grad)):
        ref = os_.rope(gy.cpu(), pos.cpu(), f, True, mscale=rot.mscale, inverse=True)
        assert bool(((got.cpu().double() - ref).abs()
                     <= bound(gy.cpu(), ref, 32, True, rot.mscale)).all())
        # differences: <dy, J dx> = <J^T dy, dx> for the linear map J, taken from the forward's
        # own outputs.  Each side sums 40*2*64 = 5120 products; every factor carries at most
        # half a bf16 step (2^-8) of its magnitude
        dx = torch.randn(t, 2, d, generator=g).to(BF16).cuda()
        jdx = rot(dx, dx, pos)[0].cpu().double()
        lhs, rhs = (gy.cpu().double() * jdx).sum(), (got.cpu().double() * dx.cpu().double()).sum()
        tol = 2.0 ** -8 * float((gy.cpu().double() * jdx).abs().sum() +
                                (got.cpu().double() * dx.cpu().double()).abs().sum())
        assert abs(float(lhs - rhs)) <= tol


def test_module_shares_positions_over_the_batch():
    g = torch.Generator().manual_seed(10)
    q, k = (torch.randn(2, 30, 3, 64, generator=g).to(BF16).cuda() for _ in range(2))
    pos = torch.arange(30, dtype=torch.int32, device="cuda")
    rot = api.Rotary(64, device="cuda")
    qo, ko = rot(q, k, pos)
    for b in range(2):
        q1, k1 = api.rope_apply(q[b], k[b], pos, rot.inv_freq)
        assert torch.equal(qo[b], q1) and torch.equal(ko[b], k1)


def test_module_takes_heads_first_broadcast_and_shifted_inputs():
    g = torch.Generator().manual_seed(12)
    n, h, d = 20, 4, 64
    rot = api.Rotary(d, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    base = torch.randn(1, h, n, d, generator=g).to(BF16).cuda()
    shared = torch.randn(1, n, 1, d, generator=g).to(BF16).cuda()  # one head for all
    flat = torch.randn(n * h * d + 3, generator=g).to(BF16).cuda()
    gy = torch.randn(1, n, h, d, generator=g).to(BF16).cuda()

    def run(leaf, view):
        leaf = leaf.clone().requires_grad_()
        x = view(leaf)
        y, _ = rot(x, x, pos)
        ref = rot(x.detach().clone().contiguous(), x.detach().clone().contiguous(), pos)[0]
        assert torch.equal(y, ref)
        y.backward(gy)
        return leaf.grad

    back = api.rope_apply(gy[0], None, pos, rot.inv_freq, inverse=True)[0]
    assert torch.equal(run(base, lambda x: x.transpose(1, 2))[0].transpose(0, 1), back)
    assert torch.equal(run(flat, lambda x: x[3:].view(1, n, h, d))[3:].view(n, h, d), back)
    # the shared head's gradient: the four heads' gradients (bf16 values) summed in bf16
    # steps: at most 3 additions, each off by half a step of a partial sum
    got = run(shared, lambda x: x.expand(1, n, h, d))[0, :, 0].double()
    mag = back.double().abs().sum(1)
    assert bool(((got - back.double().sum(1)).abs() <= 3 * 2.0 ** -8 * mag).all())
    # a single row of a wider, unaligned stride
    odd = torch.randn(2, 2 * d + 4, generator=g).to(BF16).cuda()[:1, :2 * d].view(1, 2, d)
    assert torch.equal(api.rope_apply(odd, None, pos[:1], rot.inv_freq)[0],
                       api.rope_apply(odd.clone(), None, pos[:1], rot.inv_freq)[0])


def test_replayed_graph_follows_its_positions_on_another_stream():
    q = torch.randn(9, 4, 128, generator=torch.Generator().manual_seed(11)).to(BF16).cuda()
    pos = torch.zeros(9, dtype=torch.int32, device="cuda")
    f = api.rope_inv_freq(128, device="cuda")[0]
    out = torch.empty_like(q)
    api.rope_apply(q, None, pos, f, q_out=out)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        api.rope_apply(q, None, pos, f, q_out=out)
    for p in (5, 70000):
        pos.fill_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, api.rope_apply(q, None, pos, f)[0])


def test_captured_forward_and_backward_follow_their_inputs():
    g = torch.Generator().manual_seed(13)
    rot = api.Rotary(64, interleaved=True, device="cuda")
    pos = torch.arange(15, dtype=torch.int32, device="cuda")
    q, k, gq, gk = (torch.randn(15, 2, 64, generator=g).to(BF16).cuda() for _ in range(4))
    q.requires_grad_(), k.requires_grad_()

    def step():
        out = rot(q, k, pos)
        return (*out, *torch.autograd.grad(out, (q, k), (gq, gk)))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for shift in (0, 1000):
        pos.add_(shift)
        with torch.no_grad():
            q.mul_(-1)
        gk.mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_refusals_on_device_tensors():
    q = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = api.rope_inv_freq(64, device="cuda")[0]
    for bad in (dict(positions=pos[:3]), dict(positions=pos.long()), dict(inv_freq=f.float()),
                dict(k=q[:3]), dict(k=q.float()), dict(axis_pairs=(16, 16)),
                dict(q_out=q[:, :1]), dict(q=q.transpose(0, 1)), dict(inv_freq=f.cpu())):
        args = dict(q=q, k=q, positions=pos, inv_freq=f) | bad
        with pytest.raises(ValueError):
            api.rope_apply(**args)
