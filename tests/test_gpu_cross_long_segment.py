"""A sequence so long that its part of one run takes more than the two seconds after which a wait
without progress is given up: the roles that wait for the end of the whole segment keep waiting."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from test_gpu_kv_cache import BF16

pytestmark = pytest.mark.gpu


def test_segments_longer_than_the_limit_of_waits():
    # every run gets one long segment (1 us a tile: 2.6 s) and two of a page, the second of which
    # has to wait for the long one's end; all pages are the same one
    pages, d = 2_600_000, 64
    b = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(1)
    pool = api.nvfp4_kv_pool(1, 1, d)
    kv = torch.randn(128, 2, 1, d, generator=g).to(BF16).cuda()
    api.nvfp4_kv_append_slots(kv[:, 0], kv[:, 1], torch.arange(128, device="cuda"), pool)
    table = torch.zeros(b, pages, dtype=torch.int32, device="cuda")
    lens = torch.full((b,), 128, dtype=torch.int32, device="cuda")
    lens[::3] = 128 * pages
    q = torch.randn(b, 1, d, generator=g).to(BF16).cuda()
    cu = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    o, lse = api.attn_qat_cross(q, pool, table, lens, cu)
    assert api.device_status() == 0
    # the same keys again and again: the attention over one page.  (lse: of a third of a billion
    # keys, whose sum in fp32 stops growing well before: not compared.)  Sums of p V~ and of p
    # stop together only roughly, so the long rows are only finite.
    o1, _ = api.attn_qat_cross(q, pool, table[:, :1].contiguous(), lens.clamp(max=128), cu)
    short = torch.arange(b, device="cuda") % 3 != 0
    assert torch.equal(o[short], o1[short]) and bool(torch.isfinite(o).all())
    assert bool(torch.isfinite(lse).all())
