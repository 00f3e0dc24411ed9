"""An e4m3 cache by its definition (torch on the CPU), for the tests of the
calls over it: quantisation, pages, and the values that it stands for.

Bounds of the attention over it (check_forward). With A = sum_j P_ij |V_j|:
  * P is rounded to f16 for the P V product while the row sum keeps 32 bits: off
    by at most 2^-11 of each term that is 2^-21 of the largest or more, and by
    2^-32 of the largest below that: 2^-11 A + n 2^-32 max |V| for n keys;
  * the scores are sums of d fp32 products: below 2^-12.9 for the unit normal inputs
    used here (seq_util); many rows hold q as two e4m3 parts, off by at most 2^-17 of
    the row's largest (4 here) only where it is below 2^-9 of that: for 2^-7 of the
    channels or fewer, 2^-15 * scale * sum |k| over those, below 2^-17. That moves O,
    with exponent, row sum and joining, by less than 2^-11 A;
  * O is rounded to bf16: 2^-8 |O|.
Together 2^-8 |O| + 2^-10 A + n 2^-32 max |V| (2^-11 + 2^-11 = 2^-10). LSE as in seq_util.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import seq_util as su

E4M3 = torch.float8_e4m3fn
BLOCK = 16


def exponent(amax: float) -> int:
    """The smallest e >= -64 with amax <= 448 * 2^e."""
    if amax == 0.0:
        return -64
    e = math.ceil(math.log2(amax / 448.0)) + 1
    while e > -64 and amax <= math.ldexp(448.0, e - 1):
        e -= 1
    return max(e, -64)


def codes_of(x, scale):
    """fp64 x / scale to e4m3 codes, by torch's rounding (exact quotients: scales are powers of two)."""
    y = x / scale
    return torch.where(y.isfinite(), y, math.nan).float().to(E4M3)


def scale_of(x):
    """Of rows x [n, d] (fp64): the block's scale."""
    fin = torch.where(x.isfinite(), x.abs(), 0.0)
    return math.ldexp(1.0, exponent(float(fin.max()) if fin.numel() else 0.0))


class Cache8:
    """Pages for sequences of up to `room` tokens each; nothing in them yet.
    Rows nobody wrote are NaN codes, their scales NaN, unused table entries bad."""

    def __init__(self, room, hk, d, page, seed, spare=3):
        g = su.gen(seed)
        need = [-(-n // page) for n in room]
        n = sum(need) + spare
        ids = torch.randperm(n, generator=g).tolist()
        self.page, self.hk, self.d = page, hk, d
        self.codes = [torch.full((n, page, hk, d), 0x7F, dtype=torch.uint8).view(E4M3) for _ in range(2)]
        self.scales = [torch.full((n, page // BLOCK, hk), math.nan) for _ in range(2)]
        self.table = torch.full((len(room), max(max(need), 1) + 2), -7, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
            at += m
        self.lens = [0] * len(room)

    def append(self, ks, vs):
        """By the definition; ks, vs [n, hk, d] bf16 for each sequence."""
        for b in range(len(ks)):
            n = ks[b].shape[0]
            c = self.lens[b]
            self.lens[b] = c + n
            for x, codes, scales in zip((ks[b], vs[b]), self.codes, self.scales):
                x = x.double()
                at = c
                while at < c + n:
                    end = min(c + n, at - at % BLOCK + BLOCK)
                    page, row = int(self.table[b, at // self.page]), at % self.page
                    for h in range(self.hk):
                        new = x[at - c:end - c, h]
                        sc = scale_of(new)
                        held = at % BLOCK
                        if held:
                            old = float(scales[page, row // BLOCK, h])
                            if old >= sc:
                                sc = old
                            else:
                                part = codes[page, row - held:row, h]
                                codes[page, row - held:row, h] = codes_of(part.double() * old, sc)
                        codes[page, row:row + end - at, h] = codes_of(new, sc)
                        scales[page, row // BLOCK, h] = sc
                    at = end

    def values(self, b):
        """K, V [n, hk, d] (fp64) that sequence b's rows stand for."""
        n = self.lens[b]
        out = []
        for codes, scales in zip(self.codes, self.scales):
            p = self.table[b, :-(-n // self.page)].long()
            x = codes.view(torch.uint8)[p].view(E4M3).double().view(-1, BLOCK, self.hk, self.d) * scales[p].double().view(-1, 1, self.hk, 1)
            out.append(x.reshape(-1, self.hk, self.d)[:n])
        return out

    def cuda(self):
        """k_pages, v_pages, k_scales, v_scales, and the table, on the GPU."""
        return [x.cuda() for x in self.codes + self.scales], self.table.cuda()

    def lens_k(self):
        return torch.tensor(self.lens, dtype=torch.int32)


def filled(keys, hk, d, page, seed, sigma=None):
    """A cache that holds normal K and V of these lengths (sigma: of each block of 100 keys in turn)."""
    g = su.gen(seed + 1000)
    c = Cache8(keys, hk, d, page, seed)
    ks, vs = [], []
    for n in keys:
        k, v = su.normal((n, hk, d), g).float(), su.normal((n, hk, d), g).float()
        if sigma is not None:
            s = torch.tensor([sigma[(i // 100) % len(sigma)] for i in range(n)])[:, None, None]
            v = v * s
        ks.append(k.to(torch.bfloat16))
        vs.append(v.to(torch.bfloat16))
    c.append(ks, vs)
    return c


def check_forward(o, lse, want, seqs, cu):
    o, lse = su.n64(o), su.n64(lse)
    for b, (ro, rl, big) in enumerate(want):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        go, gl = o[r0:r1], lse[:, r0:r1]
        v = seqs[b][2]
        top = float(v.abs().max()) if v.numel() else 0.0
        bound = 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * big + v.shape[0] * 2.0 ** -32 * top
        assert np.isfinite(go).all(), f"sequence {b}: O is not finite"
        bad = np.abs(go - ro) - bound
        assert go.size == 0 or (bad <= 0).all(), f"sequence {b}: O is {bad.max():.3e} beyond its bound at {np.unravel_index(bad.argmax(), bad.shape)}"
        fin = np.isfinite(rl)
        assert np.array_equal(fin, np.isfinite(gl)) and (gl[~fin] == -np.inf).all(), f"sequence {b}: empty rows"
        off = np.abs(gl[fin] - rl[fin]) - (2.0 ** -12 + 2.0 ** -22 * np.abs(rl[fin]))
        assert (off <= 0).all(), f"sequence {b}: LSE is {off.max():.3e} beyond its bound"
        assert (go[~fin.T] == 0).all(), f"sequence {b}: O of empty rows"
