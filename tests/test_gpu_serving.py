"""The packed NVFP4 linear against the float64 oracle, and the serving operators in a run:
a prompt through the training forward, its K and V into the cache, then single tokens.

Packed linear, per element: half a bf16 step of the result (2^-8 |out|), and the fp32 sum
of K exact products, whose additions are off by at most a step (2^-23) each of the running
sum: K 2^-23 sum |x~ w~| (+ the fp32 alpha, product and bias: 2^-21 of that sum and |bias|).
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api, workloads
from oracle import attention as oa
from oracle import linear as ol
from oracle import nvfp4 as onv
from oracle import serving as os_

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

SIZES = [(1, 16, 64), (1, 4608, 1536), (2, 144, 320), (5, 1536, 8960), (7, 128, 64), (8, 272, 192),
         (9, 1024, 1600), (16, 640, 4096), (17, 96, 448), (31, 2048, 256), (33, 384, 2112),
         (64, 512, 1536), (65, 208, 640), (300, 256, 2048),
         # three, five, six and seven parts of K a tile; many rows with few tiles
         (1, 5120, 1024), (4, 3200, 1600), (18, 2560, 1600), (6, 2000, 1792), (64, 1536, 1024),
         (48, 640, 1600), (3, 10256, 576),
         # more tiles of 128 weights than SMs
         (1, 19536, 64), (3, 20000, 704), (33, 39056, 576)]


def packed_bound(x, w, gx, gw, bias, ref):
    mag = onv.fq(x, gx).abs() @ onv.fq(w, gw).abs().T
    b = 0 if bias is None else bias.double().abs()
    return ref.abs() * 2.0 ** -8 + mag * (x.shape[1] * 2.0 ** -23 + 2.0 ** -21) + b * 2.0 ** -21


@pytest.mark.parametrize("m,n,k", SIZES)
def test_packed_linear_parity(m, n, k):
    inp = workloads.linear_inputs(m, n, k, seed=m + n)
    use_bias = (m + n // 16) % 2 == 1
    gw = onv.global_sf(inp.w)
    gx = None if m % 3 == 0 else 300.0
    wg = torch.tensor([gw], dtype=torch.float32, device="cuda")
    xg = None if gx is None else torch.tensor([gx], dtype=torch.float32, device="cuda")
    codes, scales = api.nvfp4_quantize_tiled(inp.w.cuda(), wg)
    xbuf = torch.full((m, k + 8), 1e30, dtype=BF16, device="cuda")  # strided rows
    xbuf[:, :k] = inp.x.cuda()
    bias = inp.bias.cuda() if use_bias else None
    ws = torch.full((api.nvfp4_linear_packed_workspace(m, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((m, n), float("nan"), dtype=BF16, device="cuda")
    args = (xbuf[:, :k], codes, scales, wg, bias, xg)
    api.nvfp4_linear_packed_fwd(*args, out=out, workspace=ws)
    assert api.device_status() == 0
    gx = onv.global_sf(inp.x) if gx is None else gx
    ref = ol.linear_fwd(inp.x, inp.w, inp.bias if use_bias else None, gx, gw)
    err = (out.cpu().double() - ref).abs()
    tol = packed_bound(inp.x, inp.w, gx, gw, inp.bias if use_bias else None, ref)
    assert bool((err <= tol).all()), float((err / tol).max())
    assert torch.equal(api.nvfp4_linear_packed_fwd(*args, workspace=ws), out)  # run to run


def test_packed_module_is_the_training_layer_s_forward():
    torch.manual_seed(3)
    lin = api.NVFP4Linear(320, 96, device="cuda")
    with torch.no_grad():
        lin.bias.normal_()
    packed = lin.pack()
    x = torch.randn(2, 3, 320, device="cuda").to(BF16)
    a, b = lin(x), packed(x)
    assert b.shape == a.shape and not b.requires_grad
    # the same exact products, summed in fp32 in another order, rounded once to bf16
    assert bool(((a - b).abs().double() <= a.abs().double() * 2.0 ** -7 + 1e-6).all())


def test_packed_module_keeps_its_types_when_the_model_changes_them():
    torch.manual_seed(4)
    packed = api.NVFP4Linear(128, 64, device="cuda").pack()
    packed.input_global_sf = torch.tensor([200.0], device="cuda")
    x = torch.randn(3, 128, device="cuda").to(BF16)
    before = packed(x)
    for change in (lambda m: m.to(BF16), lambda m: m.half(), lambda m: m.float()):
        assert torch.equal(change(packed)(x), before)


def test_packed_module_takes_any_layout():
    torch.manual_seed(5)
    packed = api.NVFP4Linear(128, 64, device="cuda").pack()
    x = torch.randn(6, 128, device="cuda").to(BF16)
    for view in (x.t().contiguous().t(), x[:1].expand(6, 128), x[::2],
                 torch.cat([x.new_zeros(1), x.flatten()])[1:].view(6, 128),
                 torch.cat([x, x[:, :3]], 1)[:, :128], torch.cat([x, x[:, :3]], 1)[:1, :128]):
        assert torch.equal(packed(view), packed(view.clone(memory_format=torch.contiguous_format)))


def test_packed_linear_unit_weight_scale_and_zero_input():
    w = workloads.random_matrix(64, 128, seed=4, scale=2.0)
    codes, scales = api.nvfp4_quantize_tiled(w.cuda())
    x = workloads.random_matrix(3, 128, seed=5)
    x[1] = 0
    xg = torch.ones(1, device="cuda")
    out = api.nvfp4_linear_packed_fwd(x.cuda(), codes, scales, None, x_global_sf=xg)
    ref = ol.linear_fwd(x, w, None, 1.0, 1.0)
    assert bool(((out.cpu().double() - ref).abs() <= packed_bound(x, w, 1.0, 1.0, None, ref)).all())
    assert not bool(out[1].any())
    z = api.nvfp4_linear_packed_fwd(torch.zeros_like(x).cuda(), codes, scales)
    assert not bool(z.any())


def test_packed_linear_graphs_share_a_workspace():
    inp = workloads.linear_inputs(4, 256, 1024, seed=6)
    codes, scales = api.nvfp4_quantize_tiled(inp.w.cuda())
    xs = [inp.x.cuda(), inp.x.cuda().neg()]
    xg = torch.tensor([200.0], device="cuda")
    ws = torch.empty(api.nvfp4_linear_packed_workspace(4, 256, 1024), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(4, 256, dtype=BF16, device="cuda") for _ in xs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for x, o in zip(xs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            api.nvfp4_linear_packed_fwd(x, codes, scales, x_global_sf=xg, out=o, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        assert torch.equal(o, api.nvfp4_linear_packed_fwd(x, codes, scales, x_global_sf=xg))
    assert torch.equal(outs[0], -outs[1])


def test_packed_linear_refusals():
    w = torch.zeros(32, 128, dtype=BF16, device="cuda")
    codes, scales = api.nvfp4_quantize_tiled(w)
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    for bad in (dict(x=x[:, :64]), dict(x=x.float()), dict(codes=codes[:, :32]), dict(scales=scales[:-1]),
                dict(bias=torch.zeros(16, dtype=BF16, device="cuda")), dict(out=x),
                dict(codes=codes.cpu()), dict(x=x.t())):
        a = dict(x=x, codes=codes, scales=scales, bias=None, out=None) | bad
        with pytest.raises(ValueError):
            api.nvfp4_linear_packed_fwd(a["x"], a["codes"], a["scales"], bias=a["bias"], out=a["out"])


def test_prompt_then_single_tokens():
    """One attention layer: QKV by the packed linear, rotary positions, causal training
    forward over the prompt and its append, then five single tokens.  Every step's output
    is held to the float64 causal oracle on the bf16 q, k, v that the GPU produced, with the
    decode bounds of test_gpu_kv_cache.py, and to the training forward's own rows."""
    h, d, n, steps = 4, 64, 200, 5
    torch.manual_seed(7)
    lin = api.NVFP4Linear(256, 3 * h * d, device="cuda").pack()
    lin.input_global_sf = torch.tensor([2688.0 / 5], device="cuda")
    rot = api.Rotary(d, device="cuda")
    x = torch.randn(n + steps, 256, device="cuda").to(BF16)
    pool = api.nvfp4_kv_pool(5, h, d)
    table = torch.tensor([[3, 1, 4]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n + steps, dtype=torch.int32, device="cuda")

    def project(rows):
        qkv = lin(x[rows]).view(-1, 3, h, d)
        q, k = rot(qkv[:, 0], qkv[:, 1], pos[rows])
        return q, k, qkv[:, 2]

    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q, k, v = project(slice(0, n))
    api.nvfp4_kv_append(k, v, lens, table, pool, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    rows, ls, qs, ks, vs = [], [], [q], [k], [v]
    for i in range(steps):
        q, k, v = project(slice(n + i, n + i + 1))
        lens += 1
        api.nvfp4_kv_append(k, v, lens, table, pool)
        o, lse = api.attn_qat_decode(q, pool, table, lens)
        rows.append(o[0])
        ls.append(lse[0])
        for lst, t in zip((qs, ks, vs), (q, k, v)):
            lst.append(t)
    q, k, v = (torch.cat(t).unsqueeze(0).contiguous() for t in (qs, ks, vs))
    _, o_hp, stats = api.attn_qat_fwd_hp(q, k, v, causal=True)
    assert api.device_status() == 0
    want = oa.attn_fwd_hp(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, True)[0, n:]
    _, lse_ref, _ = oa.attn_fwd(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, True)
    ref = os_.decode(q[0, n:].cpu(), pool.cpu(), table.cpu().expand(steps, -1),
                     list(range(n + 1, n + steps + 1)), d ** -0.5)
    assert torch.allclose(ref[0], want, atol=1e-12)  # the cache holds the forward's K~, V~
    tol = want.abs() * 2.0 ** -8 + ref[2] * 2.0 ** -10 + (n + steps) * 2.0 ** -25 * 8 + \
        2 * ref[2] * ref[3][..., None] * 2.0 ** -16
    got = torch.stack(rows).cpu().double()
    assert bool(((got - want).abs() <= tol).all())
    assert bool(((got - o_hp[0, n:].cpu().double()).abs() <= 2 * tol).all())
    got_l = torch.stack(ls).cpu().double()
    assert bool(((got_l - lse_ref[0, :, n:].T).abs() <= ref[3] * 2.0 ** -16 + 2.0 ** -18).all())
    assert bool(((got_l - stats[0, :, 0, n:].T.cpu().double()).abs() <= 2e-3).all())


def test_captured_step_between_other_kernels():
    """A decode step captured between ordinary torch kernels (the calls' launches may come up
    early, behind whatever precedes them): the replay equals the eager step, and weights
    repacked just before the linear are the ones it uses."""
    h, d, hidden = 4, 64, 256
    torch.manual_seed(8)
    w = (torch.randn(3 * h * d, hidden, device="cuda") * 0.06).to(BF16)
    x = torch.zeros(2, hidden, dtype=BF16, device="cuda")
    src = torch.randn(2, hidden, device="cuda").to(BF16)
    gain = torch.ones((), dtype=BF16, device="cuda")
    xg = torch.tensor([500.0], device="cuda")
    f = api.rope_inv_freq(d, device="cuda")[0]
    pool = api.nvfp4_kv_pool(4, h, d)
    table = torch.tensor([[0, 2], [3, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 126], dtype=torch.int32, device="cuda")
    out = torch.zeros(2, h * d, device="cuda")

    def step():
        lens.add_(1)
        x.copy_(src * 0.5)
        codes, scales = api.nvfp4_quantize_tiled(w * gain)
        qkv = api.nvfp4_linear_packed_fwd(x, codes, scales, x_global_sf=xg).view(2, 3, h, d)
        q, k = api.rope_apply(qkv[:, 0], qkv[:, 1], lens - 1, f)
        api.nvfp4_kv_append(k, qkv[:, 2], lens, table, pool)
        o, lse = api.attn_qat_decode(q, pool, table, lens)
        out.copy_(o.view(2, -1).float() + lse.mean())

    step()
    eager = []
    state = (pool.clone(), lens.clone())
    for i in range(3):
        gain.fill_(1.0 + i)
        step()
        eager.append(out.clone())
    pool.copy_(state[0])
    lens.copy_(state[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(3):
        gain.fill_(1.0 + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])
    assert api.device_status() == 0
