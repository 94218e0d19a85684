"""The largest calls of attn_qat_decode: a run of tiles is counted in 31 bits, so that more of
them are refused on the host."""
import pytest

from nvfp4_fake_quant_gb300 import _lib
from nvfp4_fake_quant_gb300 import build as nvbuild

UNSUPPORTED, WORKSPACE = 2, 3
A = 0x100000
MOST = 0x7FFFFFFF // 128  # pages of a sequence


@pytest.mark.parametrize("b,h,hkv,d,pages,runs", [
    (1, 65535, 65535, 64, MOST, 608), (1, 65535, 65535, 128, MOST, 456),
    (1, 65535, 4369, 128, MOST, 304), (4096, 32768, 32768, 64, 1 << 14, 608)])
def test_runs_past_31_bits_are_refused(b, h, hkv, d, pages, runs):
    lib = _lib.load(nvbuild.build())
    need = lib.attn_qat_decode_workspace(b, h, hkv, d, pages)

    def call(pages):
        return lib.attn_qat_decode(A, h * d, A, 8, A, pages, pages, A, b, h, hkv, d, 0.1, 0, 0,
                                   A + (1 << 40), None, A, need - 1, None)
    groups = h // hkv
    groups = -(-groups // (16 if groups > 8 else 8))
    refused = b * hkv * groups * pages // runs >= 2 ** 31 - 1
    assert call(pages) == (UNSUPPORTED if refused else WORKSPACE)
    fits = (2 ** 31 - 1) * runs // (b * hkv * groups) - 1  # the checks behind this one speak
    assert call(min(fits, pages)) == WORKSPACE
