"""The 8-bit cache in 64 bits: inputs and references of its tests (torch on the CPU)."""
from __future__ import annotations

import math

import torch

PAGE = 16
NAN_CODE = 0x7F


def e4m3_values():
    """The value of each of the 256 codes, from the format's definition (float64)."""
    vals = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v = math.nan
        elif e == 0:
            v = m / 8 * 2.0 ** -6
        else:
            v = (1 + m / 8) * 2.0 ** (e - 7)
        vals.append(-v if s else v)
    return torch.tensor(vals, dtype=torch.float64)


VALUES = e4m3_values()
_POS = VALUES[:127]  # 0 .. 448, ascending


def encode(x):
    """float64 -> codes (uint8), nearest value, ties to the even code; |x| up to 464
    (which still rounds to 448); NaN and beyond -> the NaN code."""
    a = x.abs()
    hi = torch.searchsorted(_POS, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(torch.isfinite(x) & (a <= 464.0), code, torch.tensor(NAN_CODE))
    neg = torch.signbit(x) & torch.isfinite(x)
    return (code + 128 * neg.long()).to(torch.uint8)


def decode(codes):
    return VALUES[codes.long()]


def page_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s (python floats)."""
    if not amax > 0:
        return 2.0 ** -126
    s = 2.0 ** max(-126, math.ceil(math.log2(amax / 448)) - 2)
    while amax > 448 * s:
        s *= 2
    return s


def append(codes, scales, rows, table, pos, valid):
    """The definition of storing rows [B, n, Hkv, d] (float64) in codes (uint8 [NB, Hkv,
    16, d]) and scales (float32 [NB, Hkv]), page by page, in place."""
    NB = codes.shape[0]
    for b in range(rows.shape[0]):
        p = pos[b]
        while p < pos[b] + valid[b]:
            lp, s0 = p // PAGE, p % PAGE
            s1 = min(PAGE, s0 + pos[b] + valid[b] - p)
            blk = int(table[b][lp])
            if 0 <= blk < NB:
                for g in range(rows.shape[2]):
                    x = rows[b, p - pos[b]:p - pos[b] + s1 - s0, g]
                    fin = x[torch.isfinite(x)].abs()
                    amax = float(fin.max()) if fin.numel() else 0.0
                    s = page_scale(amax)
                    was = float(scales[blk, g])
                    if s0 > 0:
                        # the comparison is in fp32, as the scale is
                        keep = was != 0 and torch.tensor(amax, dtype=torch.float32) <= \
                            scales[blk, g] * torch.tensor(448.0)
                        if bool(keep):
                            s = was
                        else:
                            codes[blk, g, :s0] = encode(decode(codes[blk, g, :s0]) * (was / s))
                    codes[blk, g, s0:s1] = encode(torch.where(torch.isfinite(x), x / s, math.nan))
                    scales[blk, g] = s
            p += s1 - s0


def rows_of(codes, scales, table_row, j):
    """Rows at positions j (int64 tensor): float64 [n, Hkv, d]."""
    blk = torch.as_tensor(table_row).long()[j // PAGE]
    return decode(codes[blk, :, j % PAGE]) * scales[blk].double()[:, :, None]


def softmax_av(z, v):
    """(softmax(z) v, softmax(z) |v|) of one row; zeros for an empty list."""
    if z.numel() == 0:
        return torch.zeros(v.shape[1], dtype=torch.float64), torch.zeros(v.shape[1], dtype=torch.float64)
    p = torch.softmax(z, 0)
    return p @ v, p @ v.abs()


class Cache:
    """A random 8-bit cache: every slot that no sequence uses holds NaN codes, every page
    that none uses has a NaN scale (nothing of either may reach a result)."""

    def __init__(self, lengths, Hkv, d, seed, power_of_two=True, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lengths = list(lengths)
        nblk = [-(-x // PAGE) for x in lengths]
        NB = sum(nblk) + spare
        width = max(1, max(nblk)) + 1
        perm = torch.randperm(NB, generator=g)
        self.table = torch.full((len(lengths), width), -1, dtype=torch.int32)
        self.codes, self.scales = [], []
        for kv in range(2):
            c = torch.full((NB, Hkv, PAGE, d), NAN_CODE, dtype=torch.uint8)
            s = torch.full((NB, Hkv), math.nan, dtype=torch.float32)
            self.codes.append(c)
            self.scales.append(s)
        first = 0
        for b, x in enumerate(lengths):
            for lp in range(nblk[b]):
                blk = int(perm[first + lp])
                self.table[b, lp] = blk
                n = min(PAGE, x - lp * PAGE)
                for kv in range(2):
                    v = torch.randn((Hkv, n, d), generator=g, dtype=torch.float64) * 60.0
                    self.codes[kv][blk, :, :n] = encode(v.clamp(-448, 448))
                    e = torch.randint(-8, -4, (Hkv,), generator=g).double()
                    sc = torch.exp2(e)
                    if not power_of_two:
                        sc = sc * (1 + torch.rand((Hkv,), generator=g, dtype=torch.float64))
                    self.scales[kv][blk] = sc.float()
            first += nblk[b]
        self.gen = g

    def cuda(self):
        """(k_cache, v_cache, k_scale, v_scale, block_table) on the GPU."""
        return (self.codes[0].cuda().view(torch.float8_e4m3fn),
                self.codes[1].cuda().view(torch.float8_e4m3fn),
                self.scales[0].cuda(), self.scales[1].cuda(), self.table.cuda())

    def kv(self, b, j):
        return (rows_of(self.codes[0], self.scales[0], self.table[b], j),
                rows_of(self.codes[1], self.scales[1], self.table[b], j))


# Bounds of a result against the definition.  bf16 outputs: half a step of bf16 (2^-8 of
# the value) and, before it, the rounding of the probabilities (at worst 2^-11 of each)
# and of the fp32 sums and exponentials (below 2^-12 of the sum of magnitudes for the
# sizes here): 2^-10 of sum_j p_j |v_j|.
def out_bound(ref, mag):
    return 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag + 1e-30


# fp32 logits: d products added in fp32 (d + 1 roundings of 2^-24 at most: 2^-16 of the
# sum of magnitudes covers d = 128 twice over) and the query held exactly to 2^-21 of its
# row's largest value.
def logit_bound(q, k, scale):
    return scale * (2.0 ** -16 * (k.abs() @ q.abs()) + 2.0 ** -20 * q.abs().max() * k.abs().sum(-1)) + 1e-30
