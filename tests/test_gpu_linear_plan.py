"""The packed NVFP4 linear of few rows in each of its layouts, against the float64 oracle
with the bound of test_gpu_serving.py: half a bf16 step of the result, 2^-8 |out|, and the
fp32 sum of K exact products, K 2^-23 sum |x~ w~| (+ alpha, product and bias: 2^-21 of that
sum and |bias|).
"""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api, workloads
from oracle import linear as ol
from oracle import nvfp4 as onv
from test_linear_plan import LAYOUTS, plan

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def sum_bound(x, w, gx, gw):
    """The bound without the result's rounding; x, w: the columns that are not zero in either."""
    mag = onv.fq(x, gx).abs() @ onv.fq(w, gw).abs().T
    return mag * (x.shape[1] * 2.0 ** -23 + 2.0 ** -21)


def guarded_workspace(m, n, k, guard=4096):
    """(workspace of exactly the size asked for, the buffer around it)."""
    need = api.nvfp4_linear_packed_workspace(m, n, k)
    buf = torch.full((need + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[guard:guard + need], buf


def test_scales_of_x_past_31_bits_of_offset():
    """K a little over 2^29: x's scales are 4 bytes an element of K, so those of the last
    columns lie past 2^31.  All but four groups of 64 columns are zero."""
    m, n, k = 2, 16, 2 ** 29 + 320
    at = [0, 2 ** 29 - 64, 2 ** 29, k - 64]
    inp = workloads.linear_inputs(m, n, 64 * len(at), seed=31)
    gx, gw = 300.0, onv.global_sf(inp.w)
    xg, wg = (torch.tensor([g], dtype=torch.float32, device="cuda") for g in (gx, gw))
    small_codes, small_scales = api.nvfp4_quantize_tiled(inp.w.cuda(), wg)
    x = torch.zeros(m, k, dtype=BF16, device="cuda")
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(k // 64 * 512, dtype=torch.uint8, device="cuda")
    small_scales = small_scales.flatten()
    for i, c in enumerate(at):
        x[:, c:c + 64] = inp.x[:, 64 * i:64 * i + 64].cuda()
        codes[:, c // 2:c // 2 + 32] = small_codes[:, 32 * i:32 * i + 32]
        scales[c // 64 * 512:c // 64 * 512 + 512] = small_scales[512 * i:512 * i + 512]
    ws, buf = guarded_workspace(m, n, k)
    out = api.nvfp4_linear_packed_fwd(x, codes, scales, wg, None, xg, workspace=ws)
    assert api.device_status() == 0
    assert bool((buf[:4096] == 0xA5).all()) and bool((buf[-4096:] == 0xA5).all())
    ref = ol.linear_fwd(inp.x, inp.w, None, gx, gw)
    err = (out.cpu().double() - ref).abs()
    # the other columns' products are zero and add nothing to the sum's error
    tol = ref.abs() * 2.0 ** -8 + sum_bound(inp.x, inp.w, gx, gw)
    assert bool((err <= tol).all())


@pytest.mark.parametrize("case", LAYOUTS, ids=lambda c: "x".join(map(str, c[:3])))
@pytest.mark.parametrize("given_scale", [True, False])
def test_parity_in_every_layout(case, given_scale):
    """The layout is the one that the size is there for, on this device too.  The weight's rows
    are 144 different ones in an order that no two tiles share."""
    m, n, k, split, fused, stages, rounds, crowded = case
    p = plan(m, n, k)
    assert (p["split"], p["fused"], p["stages"], -(-p["part"] // p["stages"])) == \
        (split, fused, stages, rounds)
    inp = workloads.linear_inputs(m, 144, k, seed=m + n + k)
    rows = torch.randint(0, 144, (n,), generator=torch.Generator().manual_seed(n))
    rows[:min(n, 144)] = torch.arange(min(n, 144))
    gw = onv.global_sf(inp.w[rows])
    gx = 300.0 if given_scale else onv.global_sf(inp.x)
    wg, xg = (torch.tensor([g], dtype=torch.float32, device="cuda") for g in (gw, gx))
    codes, scales = api.nvfp4_quantize_tiled(inp.w[rows].cuda(), wg)
    bias = inp.bias[rows].cuda() if given_scale else None
    ws, buf = guarded_workspace(m, n, k)
    ws.fill_(0xFF)
    obuf = torch.full((m * n + 64,), float("nan"), dtype=BF16, device="cuda")
    out = obuf[32:-32].view(m, n)
    args = (inp.x.cuda(), codes, scales, wg, bias, xg if given_scale else None)
    api.nvfp4_linear_packed_fwd(*args, out=out, workspace=ws)
    assert api.device_status() == 0
    assert bool((buf[:4096] == 0xA5).all()) and bool((buf[-4096:] == 0xA5).all())
    assert bool(obuf[:32].isnan().all()) and bool(obuf[-32:].isnan().all())
    ref = ol.linear_fwd(inp.x, inp.w, None, gx, gw)[:, rows]
    tol = sum_bound(inp.x, inp.w, gx, gw)[:, rows]
    if given_scale:
        b = inp.bias.double()[rows]
        ref = ref + b
        tol = tol + b.abs() * 2.0 ** -21
    tol = tol + ref.abs() * 2.0 ** -8
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert torch.equal(api.nvfp4_linear_packed_fwd(*args, workspace=ws), out)  # run to run
