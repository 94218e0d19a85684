"""Rows without keys among others, in sequences of every length: each row is written once, as 0 and
-inf, and nothing else changes."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from test_gpu_cross import ints, offsets
from test_gpu_kv_cache import BF16, make_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,most,h,d", [(1, 5000, 3, 64), (700, 1, 2, 128), (3000, 2, 1, 64),
                                        (40, 1500, 4, 64), (65535, 1, 1, 64)])
@pytest.mark.parametrize("share", [1.0, 0.5])
def test_rows(b, most, h, d, share):
    g = torch.Generator().manual_seed(b)
    toks = [1] * b if most == 1 else torch.randint(0, most + 1, (b,), generator=g).tolist()
    first = 3
    cu, t = offsets(toks, first), sum(toks) + 10
    lens = (torch.rand(b, generator=g) >= share).int() * 130
    pool = make_pool(3, 1, d, g).cuda()
    table = torch.randint(0, 3, (b, 2), generator=g).int().cuda()
    q = torch.randn(t, h, d, generator=g).to(BF16).cuda()
    o = torch.full((t, h, d), float("nan"), dtype=BF16, device="cuda")
    lse = torch.full((t, h), float("nan"), device="cuda")
    api.attn_qat_cross(q, pool, table, lens.cuda(), ints(cu), o=o, lse=lse)
    seen = torch.zeros(t, dtype=torch.bool)
    seen[first:cu[-1]] = torch.repeat_interleave(lens > 0, torch.tensor(toks))
    seen = seen.cuda()
    assert not bool(o[~seen].any()) and bool((lse[~seen] == -float("inf")).all())
    assert bool(torch.isfinite(o[seen]).all()) and bool(torch.isfinite(lse[seen]).all())
    # rows that see keys: as in a call without the others
    only = lens > 0
    if bool(only.any()):
        cu2 = offsets([n for n, k in zip(toks, only.tolist()) if k])
        o2, lse2 = api.attn_qat_cross(q[seen], pool, table[only.cuda()], lens[only].cuda(), ints(cu2))
        assert torch.equal(o[seen], o2) and torch.equal(lse[seen], lse2)
    assert api.device_status() == 0
