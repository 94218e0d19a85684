"""Serving and training calls on several streams at once, kernels that hold tensor memory in
clusters and without beside one another: every result is what the call gives alone."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api, workloads

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def linear(m, n, k, seed):
    inp = workloads.linear_inputs(m, n, k, seed=seed)
    codes, scales = api.nvfp4_quantize_tiled(inp.w.cuda())
    x, xg = inp.x.cuda(), torch.tensor([200.0], device="cuda")
    return lambda: (api.nvfp4_linear_packed_fwd(x, codes, scales, x_global_sf=xg),)


def decode(h, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randn(640, hkv, d, generator=g).to(BF16).cuda() for _ in range(2)]
    pool = api.nvfp4_kv_pool(5, hkv, d)
    table = torch.tensor([[3, 1, 4, 0, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([640], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 640], dtype=torch.int32, device="cuda")
    api.nvfp4_kv_append(*kv, lens, table, pool, cu)
    q = torch.randn(24, h, d, generator=g).to(BF16).cuda()
    tables = table.expand(24, -1).contiguous()
    lens = torch.arange(17, 641, 26, dtype=torch.int32, device="cuda")
    return lambda: api.attn_qat_decode(q, pool, tables, lens)


def attention(d, seed):
    inp = workloads.attn_inputs(1, 1024, 1024, 4, d, seed=seed)
    q, k, v, do = (t.cuda() for t in (inp.q, inp.k, inp.v, inp.do))

    def call():
        o, stats = api.attn_qat_fwd(q, k, v, inp.scale)
        return (o, *api.attn_qat_bwd(q, k, v, o, stats, do, inp.scale))
    return call


def test_calls_on_their_own_streams():
    calls = [linear(1, 4608, 1536, 1), linear(5, 1536, 8960, 2), linear(64, 2048, 2048, 3),
             linear(300, 512, 1024, 4), linear(12, 8320, 1024, 5), decode(8, 2, 64, 6),
             decode(32, 2, 64, 7), decode(8, 8, 128, 8), attention(64, 9), attention(128, 10)]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(12):
        for i, (call, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(call())
    torch.cuda.synchronize()
    assert api.device_status() == 0
    for results, w in zip(got, want):
        assert all(torch.equal(a, b) for r in results for a, b in zip(r, w))
