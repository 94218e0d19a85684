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
