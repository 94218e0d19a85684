"""Frequencies of several position axes: one ladder by default, one per axis where inv_freq
gives it, as the docstring of api.Rotary says (the kernel replaced by the oracle, on the CPU)."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_


def test_one_ladder_or_one_per_axis(monkeypatch):
    def oracle_rope(q, k, positions, inv_freq, interleaved, axis_pairs, mscale, inverse=False):
        return tuple(os_.rope(x, positions, inv_freq, interleaved, axis_pairs, mscale, inverse)
                     for x in (q, k))
    monkeypatch.setattr(api, "rope_apply", oracle_rope)
    g = torch.Generator().manual_seed(1)
    pairs, d = (4, 6, 6), 32
    x = torch.randn(5, 2, d, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 40, (5, 3), generator=g, dtype=torch.int32)
    one = api.Rotary(d, interleaved=True, axis_pairs=pairs)(x, x, pos)[0]
    per = torch.cat([api.rope_inv_freq(2 * n)[0] for n in pairs])
    each = api.Rotary(d, interleaved=True, axis_pairs=pairs, inv_freq=per)(x, x, pos)[0]
    ladder, at = api.rope_inv_freq(d)[0], 0
    for axis, n in enumerate(pairs):  # adjacent pairs: an axis owns a slice of the head
        part = slice(2 * at, 2 * (at + n))
        own = api.rope_inv_freq(2 * n)[0]
        assert torch.equal(each[..., part], os_.rope(x[..., part], pos[:, axis], own, True))
        assert torch.equal(one[..., part],
                           os_.rope(x[..., part], pos[:, axis], ladder[at:at + n], True))
        at += n


def test_given_frequencies_go_to_the_device_and_stand_alone():
    f = api.rope_inv_freq(32)[0]
    assert api.Rotary(32, inv_freq=f, device="meta").inv_freq.device.type == "meta"
    assert api.Rotary(32, inv_freq=f).inv_freq is f
    # what would have shaped them is not dropped without a word
    with pytest.raises(ValueError, match="theta"):
        api.Rotary(32, inv_freq=f, theta=500000.0)
