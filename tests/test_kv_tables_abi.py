"""Refusals of the cache's table calls and of the append by slots: wrong sizes and pointers
return their status on the host, before any CUDA call."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import _lib, api
from nvfp4_fake_quant_gb300 import build as nvbuild

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 0x100000


@pytest.fixture(scope="module")
def lib():
    return _lib.load(nvbuild.build())


def test_extend_refusals(lib):
    def ext(new=A, lens=A, start=None, b=3, table=A, ld=4, mp=4, free=A, count=A, pages=8, t=5,
            lens_out=A, count_out=A, cu=A, pos=A, slots=A):
        return lib.nvfp4_kv_extend(new, lens, start, b, table, ld, mp, free, count, pages, t,
                                   lens_out, count_out, cu, pos, slots, None)
    for bad in (dict(new=None), dict(new=A + 2), dict(lens=None), dict(lens=A + 1),
                dict(start=A + 2), dict(b=0), dict(b=-1), dict(table=None), dict(table=A + 2),
                dict(ld=3), dict(mp=0), dict(mp=1 << 25), dict(free=None), dict(free=A + 2),
                dict(count=None), dict(count=A + 3), dict(pages=0), dict(pages=1 << 31),
                dict(t=-1), dict(lens_out=None), dict(count_out=None), dict(cu=None),
                dict(cu=A + 2), dict(pos=None), dict(pos=A + 2), dict(slots=None),
                dict(slots=A + 4)):
        assert ext(**bad) == INVALID, bad
    assert ext(b=65536) == UNSUPPORTED and ext(t=1 << 31) == UNSUPPORTED


def test_release_refusals(lib):
    def rel(done=A, lens=A, b=3, table=A, ld=4, mp=4, free=A, count=A, pages=8, lens_out=A,
            count_out=A):
        return lib.nvfp4_kv_release(done, lens, b, table, ld, mp, free, count, pages, lens_out,
                                    count_out, None)
    for bad in (dict(done=None), dict(lens=None), dict(lens=A + 2), dict(b=0), dict(table=None),
                dict(ld=3), dict(mp=0), dict(free=None), dict(count=None), dict(count=A + 2),
                dict(pages=0), dict(lens_out=None), dict(lens_out=A + 2), dict(count_out=None)):
        assert rel(**bad) == INVALID, bad
    assert rel(b=65536) == UNSUPPORTED


def test_outputs_over_other_arguments_are_refused(lib):
    """Every other argument on a range of its own, then one output at a time over another (the
    starts as the lengths that the call writes: a second kernel would read them too late)."""
    names = "new lens start table free count lens_out count_out cu pos slots".split()
    at = {n: A + 0x10000 * i for i, n in enumerate(names)}

    def ext(b=3, t=5, ld=6, **over):
        g = at | over
        return lib.nvfp4_kv_extend(g["new"], g["lens"], g["start"], b, g["table"], ld, 4, g["free"],
                                   g["count"], 8, t, g["lens_out"], g["count_out"], g["cu"],
                                   g["pos"], g["slots"], None)
    size = dict(new=12, lens=12, start=12, table=64, free=32, count=4, lens_out=12, count_out=4,
                cu=16, pos=20, slots=40)
    for out in ("lens_out", "count_out", "cu", "pos", "slots", "table"):
        for other in names:
            step = 8 if out == "slots" else 4
            last = at[other] + (size[other] - 1) // step * step  # its last word
            if other != out and not (out, other) == ("count_out", "count"):
                assert ext(**{out: last}) == INVALID, (out, other)
    assert ext(lens_out=at["lens"] + 4) == INVALID
    assert ext(start=at["lens_out"], lens=at["lens_out"]) == INVALID
    assert ext(t=0, pos=at["table"] + 8, slots=at["table"] + 16, lens_out=at["cu"]) == INVALID

    def rel(b=3, **over):
        g = at | over
        return lib.nvfp4_kv_release(g["new"], g["lens"], b, g["table"], 6, 4, g["free"], g["count"],
                                    8, g["lens_out"], g["count_out"], None)
    for over in (dict(lens_out=at["table"] + 60), dict(lens_out=at["free"]), dict(lens_out=at["new"]),
                 dict(count_out=at["free"] + 28), dict(free=at["table"] + 32), dict(free=at["lens"]),
                 dict(count_out=at["lens_out"] + 8), dict(free=at["count"] - 28)):
        assert rel(**over) == INVALID, over


def test_append_slots_refusals(lib):
    def app(k=A, ld_k=256, v=A, ld_v=256, t=3, hkv=2, d=128, slots=A, pool=A, pages=8):
        return lib.nvfp4_kv_append_slots(k, ld_k, v, ld_v, t, hkv, d, slots, pool, pages, None)
    assert app(t=0, k=None, slots=None, pool=None) == OK
    for bad in (dict(t=-1), dict(hkv=0), dict(k=None), dict(v=A + 8), dict(ld_k=248),
                dict(ld_v=260), dict(slots=None), dict(slots=A + 4), dict(pool=None),
                dict(pool=A + 8), dict(pages=0), dict(pages=1 << 31)):
        assert app(**bad) == INVALID, bad
    assert app(d=96) == UNSUPPORTED and app(hkv=65536, ld_k=1 << 24, ld_v=1 << 24) == UNSUPPORTED


def test_python_layer_refusals():
    n, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    one, free = torch.zeros(1, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.nvfp4_kv_extend(n, n, table, free, one)
    for bad in ((n[:1], n, table, free, one), (n, n[:1], table, free, one),
                (n, n, table[0], free, one), (n, n, table.long(), free, one),
                (n, n, table, free.view(1, 5), one), (n, n, table, free, n),
                (n.float(), n, table, free, one)):
        with pytest.raises(ValueError):
            api.nvfp4_kv_extend(*bad)
    for bad in (dict(tokens=-1), dict(start=one), dict(cu_tokens=n), dict(seq_lens_out=free)):
        with pytest.raises(ValueError):
            api.nvfp4_kv_extend(n, n, table, free, one, **bad)
    with pytest.raises(ValueError, match="CUDA"):
        api.nvfp4_kv_release(n.bool(), n, table, free, one)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.nvfp4_kv_append_slots(x, x, n.long(), api.nvfp4_kv_pool(1, 1, 64, device="cpu"))
