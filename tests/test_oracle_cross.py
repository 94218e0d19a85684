"""The oracle of many rows over the cache against its single-token oracle and brute force."""
import torch

from oracle import serving as os_


def _pool(pages, hkv, d, g):
    pool = torch.empty(pages, hkv, 144 * d, dtype=torch.uint8)
    for at_c, at_s in ((0, 128 * d), (64 * d, 136 * d)):
        c, s = os_.pack(torch.randn(pages, hkv, 128, d, generator=g).to(torch.bfloat16))
        pool[:, :, at_c:at_c + 64 * d], pool[:, :, at_s:at_s + 8 * d] = c.flatten(2), s.flatten(2)
    return pool


def test_attend_is_decode_row_by_row():
    g = torch.Generator().manual_seed(0)
    pool, table = _pool(5, 2, 64, g), torch.tensor([[3, 0, 4]])
    q = torch.randn(3, 6, 64, generator=g).to(torch.bfloat16)
    got = os_.attend(q, pool, [(table[0], 300)], 0.125)
    want = os_.decode(q, pool, table.expand(3, -1), [300] * 3, 0.125)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=0, atol=1e-12)


def test_attend_over_two_spans_is_one_sequence():
    """A prefix of whole pages and own tokens: the sequence whose table is both."""
    g = torch.Generator().manual_seed(1)
    pool, q = _pool(5, 1, 64, g), torch.randn(2, 2, 64, generator=g).to(torch.bfloat16)
    got = os_.attend(q, pool, [(torch.tensor([4, 1]), 256), (torch.tensor([0]), 37)], 0.2)
    want = os_.decode(q, pool, torch.tensor([[4, 1, 0]]).expand(2, -1), [293] * 2, 0.2)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=0, atol=1e-12)


def test_no_keys():
    g = torch.Generator().manual_seed(2)
    o, lse, _, _ = os_.attend(torch.randn(2, 2, 64).to(torch.bfloat16), _pool(1, 1, 64, g),
                              [(torch.tensor([0]), 0)], 0.1)
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
