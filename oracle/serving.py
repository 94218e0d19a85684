"""Oracle of the single-token serving operators and the rotary positions (TEST
INFRASTRUCTURE ONLY; see ``oracle/__init__``), float64 on the CPU.

  rope          pairs of a head turned by position * inv_freq
  cache         page records (K codes | V codes | K scales | V scales of 128 tokens
                and one head) packed from and unpacked to values
  decode        one query token per sequence over the visible cached keys, with the
                sums of magnitudes that the tests' error bounds are made of
"""
from __future__ import annotations

import torch

from .nvfp4 import E2M1_GRID, E4M3_VALUES, fake_quant, fq

F64 = torch.float64
PAGE = 128


def rope(x, positions, inv_freq, interleaved=False, axis_pairs=None, mscale=1.0, inverse=False):
    """x [T, H, D] float64-rotated; positions [T] or [T, axes]."""
    pos = positions.reshape(x.shape[0], -1).to(F64)
    pairs = inv_freq.numel()
    counts = (pairs,) if axis_pairs is None else tuple(axis_pairs)
    axis = [a for a, n in enumerate(counts) for _ in range(n)]
    ang = pos[:, axis] * inv_freq.to(F64) * (-1.0 if inverse else 1.0)
    c, s = torch.cos(ang)[:, None] * mscale, torch.sin(ang)[:, None] * mscale
    i = torch.arange(pairs)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    y = x.to(F64).clone()
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = a * c - b * s, a * s + b * c
    return y


def record_parts(pool, d):
    """K codes, V codes [pages, H, 128, D/2], K scales, V scales [pages, H, 128, D/16] (copies)."""
    c, s = PAGE * d // 2, PAGE * d // 16
    a, b, e, f = pool.cpu().split([c, c, s, s], dim=-1)
    shape = pool.shape[:2] + (PAGE, -1)
    return tuple(t.reshape(shape) for t in (a, b, e, f))


def unpack(codes, scales):
    """float64 values of packed codes [..., n/2] and E4M3 scale bytes [..., n/16]."""
    idx = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    mag = E2M1_GRID[idx & 7] * (1.0 - 2.0 * (idx >> 3).to(F64))
    s = torch.where(scales < 0x7F, E4M3_VALUES[scales.long().clamp(max=0x7E)],
                    torch.full((), float("nan"), dtype=F64))
    return (mag.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def pack(x):
    """(packed codes, scale bytes) of x [..., n] under the unit scale."""
    _, sb, codes = fake_quant(x)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sb


def visible(n, window, sinks):
    return [j for j in range(n) if window == 0 or j >= n - window or j < sinks]


def decode(q, pool, table, lens, scale, window=0, sinks=0, keep=None):
    """q [B, H, D]; returns (o, lse, mag, err_s), float64: mag[b, h, :] = sum p |v| / l and
    err_s[b, h] = scale * max_j sum_i |q_i k_ji|, the magnitudes that bound rounding errors.
    keep(b, j): False leaves out a key beyond the window's rule."""
    b, h, d = q.shape
    hkv = pool.shape[1]
    kc, vc, ks, vs = record_parts(pool, d)
    qq = fq(q)
    o = torch.zeros(b, h, d, dtype=F64)
    lse = torch.full((b, h), -float("inf"), dtype=F64)
    mag, err_s = torch.zeros(b, h, d, dtype=F64), torch.zeros(b, h, dtype=F64)
    for i in range(b):
        seen = [j for j in visible(int(lens[i]), window, sinks) if keep is None or keep(i, j)]
        if not seen:
            continue
        j = torch.tensor(seen)
        page = table[i].cpu()[j // PAGE].long()
        for hk in range(hkv):
            k = unpack(kc[page, hk, j % PAGE], ks[page, hk, j % PAGE])
            v = unpack(vc[page, hk, j % PAGE], vs[page, hk, j % PAGE])
            for g in range(h // hkv):
                hh = hk * (h // hkv) + g
                s = scale * (k @ qq[i, hh])
                p = torch.softmax(s, 0)
                o[i, hh], mag[i, hh] = p @ v, p @ v.abs()
                lse[i, hh] = torch.logsumexp(s, 0)
                err_s[i, hh] = scale * (k.abs() @ qq[i, hh].abs()).max()
    return o, lse, mag, err_s
