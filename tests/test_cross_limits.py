"""The largest sizes that attn_qat_cross takes, on both sides of the documented bounds (host only):
(T*H/Hkv/128 + B) * Hkv * max_pages < 2^34 and T*H < 2^31 - 256."""
import pytest

from nvfp4_fake_quant_gb300 import _lib
from nvfp4_fake_quant_gb300 import build as nvbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A, O, BIG = 0x100000, 1 << 46, 1 << 45


@pytest.fixture(scope="module")
def lib():
    return _lib.load(nvbuild.build())


@pytest.mark.parametrize("t,b,h,hkv,mp,fits", [
    (1, 1023, 16, 16, 1 << 20, True), (1, 1024, 16, 16, 1 << 20, False),
    (1, 1024, 16, 16, (1 << 20) - 1, True),
    (1, 1, 1024, 1024, (1 << 24) - 1, True), (128, 1, 1024, 1024, (1 << 24) - 1, False),
    (127, 1, 1024, 1024, (1 << 24) - 1, True),
    (128 * 1023, 1, 8, 8, 1 << 21, False), (128 * 1023, 1, 8, 8, (1 << 21) - 1, True),
    (128 * 1023 // 4, 1, 32, 8, 1 << 21, False), (128 * 1023 // 4 - 1, 1, 32, 8, 1 << 21, True),
    (2047, 65535, 4, 4, 65536, False), (2047, 65535, 4, 4, 65520, True),
])
def test_tiles(lib, t, b, h, hkv, mp, fits):
    assert ((t * (h // hkv) // 128 + b) * hkv * mp < 1 << 34) == fits
    assert (lib.attn_qat_cross_workspace(t, b, h, hkv, 64, mp) > 0) == fits
    if b <= 65535 and t > 1:
        st = lib.attn_qat_cross(A, h * 64, t, A, 8, A, mp, mp, A, A, b, h, hkv, 64, 0.1, O, None,
                                None, 0, None)
        assert st == (WORKSPACE if fits else UNSUPPORTED)


def test_prefix(lib):
    def need(b, s, pp):
        return lib.attn_qat_decode_prefix_workspace(b, s, 16, 16, 64, 4, pp)
    # 1024 rows of a KV head are 8 of the bound's units
    assert need(1024, 1015, 1 << 20) > 0 and need(1024, 1016, 1 << 20) == 0
    assert need(1024, 1016, (1 << 20) - 1) > 0


def test_rows(lib):
    last = ((1 << 31) - 256) // 8 - 1
    assert lib.attn_qat_cross_workspace(last, 1, 8, 8, 64, 4) > 0
    assert lib.attn_qat_cross_workspace(last + 1, 1, 8, 8, 64, 4) == 0
