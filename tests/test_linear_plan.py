"""How the packed linear of few rows lays out a call, on the host: nothing is launched."""
import ctypes

import pytest

from nvfp4_fake_quant_gb300 import _lib
from nvfp4_fake_quant_gb300 import build as nvbuild

FIELDS = ("split", "ctas", "fused", "part", "stages", "smem", "x_scales", "x_scales_end")


def plan(m, n, k):
    lib = _lib.load(nvbuild.build())
    got = (ctypes.c_int64 * len(FIELDS))()
    assert lib.nvq_selftest_linear_plan(m, n, k, ctypes.addressof(got)) == 0
    return dict(zip(FIELDS, got))


@pytest.mark.parametrize("k", [64, 1536, 2 ** 20, 2 ** 29 - 64, 2 ** 29, 2 ** 29 + 64, 2 ** 29 + 256,
                               2 ** 30 - 64, 2 ** 30])
@pytest.mark.parametrize("m", [1, 2, 17, 31])
def test_scales_of_x_stay_in_their_region(m, k):
    """Stages of 256 elements have 1 KB of scales; the furthest lies in the last stage."""
    p = plan(m, 16, k)
    assert p["x_scales"] == -(-k // 256) * 1024
    assert p["x_scales"] - 1024 < p["x_scales_end"] <= p["x_scales"]


def test_plan_refusals():
    lib = _lib.load(nvbuild.build())
    got = (ctypes.c_int64 * len(FIELDS))()
    at = ctypes.addressof(got)
    for m, n, k, out in ((0, 16, 64, at), (1, 24, 64, at), (1, 16, 32, at), (1, 16, 64, None)):
        assert lib.nvq_selftest_linear_plan(m, n, k, out) == 1
    assert lib.nvq_selftest_linear_plan(65, 16, 64, at) == 2


@pytest.mark.parametrize("m,k", [(1, 64), (5, 8960), (33, 2112), (64, 16384)])
def test_workspace_follows_from_x_alone(m, k):
    """Codes of x, its scales at a 256-byte boundary, one scalar: whatever the weights' rows
    and the device are."""
    lib = _lib.load(nvbuild.build())
    want = -(-m * k // 2 // 256) * 256 + -(-k // 256) * 1024 + 256
    for n in (16, 4608, 53248):
        assert lib.nvfp4_linear_packed_workspace(m, n, k) == want


# m, n, k and the layout each is there for: CTAs a tile, x quantized by them, stages of the
# ring, times that a CTA goes around it (rounded up), more CTAs than multiprocessors
LAYOUTS = [
    (64, 128, 32768, 4, 0, 4, 8, 0), (33, 272, 24640, 5, 0, 4, 5, 0), (1, 128, 32768, 8, 0, 4, 4, 0),
    (1, 8192, 1024, 3, 1, 2, 1, 1), (32, 10240, 8192, 2, 0, 4, 4, 1), (16, 8320, 4096, 3, 0, 4, 2, 1),
    (64, 8320, 2240, 2, 0, 2, 3, 0), (1, 7680, 5632, 3, 1, 3, 3, 1), (8, 4992, 4160, 4, 0, 4, 2, 1),
    (4, 39056, 2112, 1, 0, 4, 3, 1), (1, 19584, 1280, 1, 1, 4, 2, 1), (17, 1664, 6464, 6, 0, 4, 2, 0),
    (31, 128, 1792, 7, 0, 1, 1, 0), (31, 144, 2048, 8, 0, 1, 1, 0), (1, 128, 1600, 7, 1, 1, 1, 0),
    (1, 4992, 6464, 4, 1, 3, 3, 1), (64, 1920, 8192, 4, 0, 4, 2, 0),
]


@pytest.mark.parametrize("case", LAYOUTS, ids=lambda c: "x".join(map(str, c[:3])))
def test_layouts(case):
    m, n, k, split, fused, stages, rounds, crowded = case
    p = plan(m, n, k)
    got = (p["split"], p["fused"], p["stages"], -(-p["part"] // p["stages"]), int(p["ctas"] > 152))
    assert got == (split, fused, stages, rounds, crowded)


def test_every_plan_keeps_its_promises():
    """Over many sizes: a stage for the ring, the shared memory a block may have, two blocks an
    SM where there are more of them than fit one each, and never three (each holds half of the
    tensor memory)."""
    sms, smem = 152, 228 * 1024
    for m in (1, 3, 16, 17, 28, 32, 33, 48, 49, 64):
        for tiles in [*range(1, 50), 65, 76, 100, 152, 153, 304, 400]:
            for k in [64, *range(256, 9000, 448), 16384, 65536]:
                p = plan(m, 128 * tiles, k // 64 * 64)
                assert 1 <= p["stages"] <= p["part"] and p["split"] <= 8
                assert p["ctas"] == p["split"] * tiles
                assert p["smem"] <= 227 * 1024 and 3 * (p["smem"] + 1024) > smem
                if p["ctas"] > sms:
                    assert 2 * (p["smem"] + 1024) <= smem


@pytest.mark.parametrize("m", [1, 5, 8, 16])
@pytest.mark.parametrize("k", [2048, 8192, 28672])
def test_sixteen_clusters_of_seven_or_eight_are_not_asked_for(m, k):
    """With one CTA per SM the chip's groups of SMs hold 15 of them at once."""
    assert plan(m, 15 * 128, k)["split"] == 8
    assert plan(m, 16 * 128, k)["split"] == 6
