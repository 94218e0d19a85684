"""The packed linear reads x until its last output is written: an output over x is refused on
the host."""
import pytest

from nvfp4_fake_quant_gb300 import _lib
from nvfp4_fake_quant_gb300 import build as nvbuild

INVALID, WORKSPACE = 1, 3
A = 0x100000
BIG = 1 << 40


@pytest.mark.parametrize("m,n,k,ld", [(1, 128, 128, 128), (2, 128, 128, 128), (2, 128, 128, 256),
                                      (5, 1536, 1536, 1536), (64, 96, 4096, 4104),
                                      (65, 96, 128, 128), (300, 128, 64, 72)])
def test_output_over_x_is_refused(m, n, k, ld):
    lib = _lib.load(nvbuild.build())

    def call(x, out, ws=A, ws_bytes=BIG):
        return lib.nvfp4_linear_packed_fwd(x, ld, A, A, None, None, m, n, k, None, out, ws, ws_bytes,
                                           None)
    x_bytes, out_bytes = 2 * ((m - 1) * ld + k), 2 * m * n
    assert call(A, A) == INVALID
    assert call(A, A + x_bytes - 16) == INVALID
    assert call(A + out_bytes - 16, A) == INVALID
    # next to each other: the checks before and after this one speak
    assert call(A, A + x_bytes, ws_bytes=0) == WORKSPACE
    assert call(A + out_bytes, A, ws_bytes=0) == WORKSPACE
