"""Rows that enter a cache, the weight they gather and their eviction, in 64 bits: inputs and
references of those tests (torch on the CPU)."""
from __future__ import annotations

import math

import torch

PAGE = 16


def inv_freq(rot, theta=1e6):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))


def turned(x, weight, eps, pos, freq, interleaved, amplitude=1.0):
    """Rows x [n, H, d] (float64) normed and rotated by pos [n] (python integers or int64):
    (result, bound of the fp32 arithmetic before the result is rounded)."""
    y = x.clone()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    # fp32: the sum of 128 squares, 1 / sqrt and two products: below 2^-20 of the value
    off = 2.0 ** -20 * y.abs()
    half = freq.numel()
    if half:
        i = torch.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = (torch.as_tensor(pos).double()[:, None] * freq).remainder(2 * math.pi)[:, None]
        c, s = amplitude * torch.cos(angle), amplitude * torch.sin(angle)
        y0, y1 = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = y0 * c - y1 * s, y1 * c + y0 * s
        # ... the angle to 2^-24 of half a turn (pi 2^-24 < 2^-22), sin and cos to 2^-22, three
        # roundings: with the norm's 2^-20, below 2^-19 of the sum of magnitudes
        both = 2.0 ** -19 * abs(amplitude) * (y0.abs() + y1.abs())
        off[..., a], off[..., b] = both, both
    return y, off


def bf16_bound(ref, off):
    """A result in bf16: half a step of bf16 (2^-8 of the value) and the arithmetic's part."""
    return 2.0 ** -8 * ref.abs() + 1.01 * off + 2.0 ** -130


def tables(lengths, gen, spare=2, width=None, first=None):
    """A block table over shuffled blocks (-1: unused) for sequences of these lengths, and the
    blocks that are left over."""
    nblk = [-(-x // PAGE) for x in lengths]
    NB = sum(nblk) + spare
    ids = torch.randperm(NB, generator=gen) if first is None else first
    width = width or max(1, max(nblk)) + 1
    t = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        t[b, :n] = ids[at:at + n].int()
        at += n
    return t, ids[at:]


def accumulated(weights, logits, block_logits, rows, prefix, G):
    """weights [B, Hkv, W] (float64) after the call, and its bound.  block_logits[b][c]: [Hq, r_c + 1]."""
    out, bound = weights.clone(), 2.0 ** -24 * weights.abs()
    for b, P in enumerate(prefix):
        for c, r in enumerate(rows):
            if r < 0 or P == 0:
                continue
            z = torch.cat([logits[b, c, :, :P].double(), block_logits[b][c]], 1)
            m = z.max(1, keepdim=True).values
            p = torch.softmax(z, 1)[:, :P]
            # exponent in fp32: 2^-23 of m - z for the difference and the product with log2 e;
            # exponentials 2^-22, the sum and its reciprocal below 2^-20
            off = torch.where(p > 0, p * (2.0 ** -19 + 2.0 ** -22 * (m - z[:, :P])), 0.0) + 2.0 ** -120
            out[b, :, :P] += p.view(-1, G, P).sum(1)
            bound[b, :, :P] += off.view(-1, G, P).sum(1)
    return out, bound + 2.0 ** -22 * out.abs()
