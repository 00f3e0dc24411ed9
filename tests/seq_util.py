"""Inputs, the 64-bit reference and the bounds shared by the tests of the
calls on sequences of different lengths.

The reference is the oracle's dense attention, one sequence at a time.

Bounds. An O element is sum_j P_ij V_j; with A = sum_j P_ij |V_j| (the same
attention of |V|):
  * P is rounded to bf16 for the P V product while the row sum keeps 32 bits:
    off by at most 2^-8 of each term, so 2^-8 A;
  * O is rounded to bf16: 2^-8 |O|;
  * the scores are sums of d fp32 products: off by at most (d + 2) 2^-24
    scale sum_c |q_c k_c|, which for d = 128 and the unit normal inputs used
    here (scale sum |q k| < 16) is below 2^-12.9; exponent and row sum together
    change O by at most twice that, and O's joining by fp32 roundings more:
    2^-11 A covers them.
LSE is off by at most the scores' own 2^-12.9 and the row sum's rounding (at
most n / 8 adds of 2^-24 for n keys: below 2^-13 for n < 16384): 2^-12 + 2^-22
|lse|.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import attn_ref


def starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32)


def normal(shape, g, sigma=1.0):
    return (torch.randn(shape, generator=g, dtype=torch.float32) * sigma).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def n64(t):
    return t.detach().double().cpu().numpy()


def window_of(causal, window):
    return (-1 if window is None else window[0], 0 if causal else (-1 if window is None else window[1]))


def reference(seqs, scale, causal=False, window=None):
    """seqs: (q [n, Hq, d], k [m, Hkv, d], v) per sequence, tensors. Returns
    per sequence (O, LSE [Hq, n], A) in 64 bits."""
    out = []
    for q, k, v in seqs:
        n, hq, d = q.shape
        if n == 0:
            out.append((np.zeros((0, hq, d)), np.zeros((hq, 0)), np.zeros((0, hq, d))))
        elif k.shape[0] == 0:
            out.append((np.zeros((n, hq, d)), np.full((hq, n), -np.inf), np.zeros((n, hq, d))))
        else:
            a = [n64(x)[None] for x in (q, k, v)]
            o, lse = attn_ref.forward(*a, scale, causal, window=window)
            big, _ = attn_ref.forward(a[0], a[1], np.abs(a[2]), scale, causal, window=window)
            out.append((o[0], lse[0], big[0]))
    return out


def check_forward(o, lse, want, cu):
    """o [total, Hq, d], lse [Hq, total] (tensors) against reference()."""
    o, lse = n64(o), n64(lse)
    for b, (ro, rl, big) in enumerate(want):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        go, gl = o[r0:r1], lse[:, r0:r1]
        assert np.isfinite(go).all(), f"sequence {b}: O is not finite"
        bound = 2.0 ** -8 * (big + np.abs(ro)) + 2.0 ** -11 * big
        bad = np.abs(go - ro) - bound
        assert (bad <= 0).all(), f"sequence {b}: O is {bad.max():.3e} beyond its bound at {np.unravel_index(bad.argmax(), bad.shape)}"
        fin = np.isfinite(rl)
        assert np.array_equal(fin, np.isfinite(gl)) and (gl[~fin] == -np.inf).all(), f"sequence {b}: empty rows"
        off = np.abs(gl[fin] - rl[fin]) - (2.0 ** -12 + 2.0 ** -22 * np.abs(rl[fin]))
        assert (off <= 0).all(), f"sequence {b}: LSE is {off.max():.3e} beyond its bound"
        # rows without a key
        assert (go[~fin.T] == 0).all(), f"sequence {b}: O of empty rows"


def reference_backward(seqs, douts, os, scale, causal=False, window=None):
    """Per sequence the oracle's (dQ, dK, dV) in 64 bits with elementwise
    bounds for a backward pass that was given the bf16 outputs `os`.

    Bounds. dV_j = sum_i P_ij dO_i, dS_ij = P_ij (dP_ij - D_i), dQ_i = scale sum_j
    dS_ij K_j, dK_j = scale sum_i dS_ij Q_i, with P and dS rounded to bf16 before the
    products (2^-8 of each term) and the results rounded to bf16 (2^-8). P
    itself comes from 32-bit scores and the 32-bit LSE: off by 2^-11 of itself
    (scores below 2^-12.9, see the module's notes, and as much again for LSE);
    dP and D are sums of d fp32 products, off by (d + 2) 2^-24 sum |dO_c V_c| each.
    D is formed from the bf16 O: dS moves by P_ij |dO_i . (O_bf16 - O)_i|.
    With R_ij = P_ij (|dP_ij| + |D_i|) and E_ij = P_ij (|dO_i . dO_err| + 2^-15 (A_i)),
    A_i = sum_c |dO_ic| max_j |V_jc|, the bounds are the products of (2^-8 + 2^-10) R + E
    with |K| and |Q|."""
    out = []
    for (q, k, v), do, o in zip(seqs, douts, os):
        n, hq, d = q.shape
        m, hk, _ = k.shape
        G = hq // hk
        Q, K, V, DO, O = (n64(x) for x in (q, k, v, do, o))
        dq, dk, dv = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(V)
        bq, bk, bv = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(V)
        if n and m:
            see = attn_ref.visible_mask(np.arange(n), n, m, causal, window)
            for h in range(hq):
                g = h // G
                s = np.where(see, scale * Q[:, h] @ K[:, g].T, -np.inf)
                top = s.max(1, keepdims=True)
                e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
                l = e.sum(1, keepdims=True)
                p = e / np.where(l > 0, l, 1.0)
                ex = p @ V[:, g]
                dp = DO[:, h] @ V[:, g].T
                D = (DO[:, h] * ex).sum(1, keepdims=True)
                ds = p * (dp - D)
                dq[:, h] = scale * ds @ K[:, g]
                dk[:, g] += scale * ds.T @ Q[:, h]
                dv[:, g] += p.T @ DO[:, h]
                R = p * (np.abs(dp) + np.abs(D))
                err = np.abs((DO[:, h] * (O[:, h] - ex)).sum(1, keepdims=True))
                A = (np.abs(DO[:, h]) * np.abs(V[:, g]).max(0)).sum(1, keepdims=True)
                t = (2.0 ** -8 + 2.0 ** -10) * R + p * (err + 2.0 ** -15 * A)
                a = abs(scale)
                bq[:, h] = a * t @ np.abs(K[:, g])
                bk[:, g] += a * t.T @ np.abs(Q[:, h])
                bv[:, g] += (2.0 ** -8 + 2.0 ** -10) * p.T @ np.abs(DO[:, h])
        for x, b in ((dq, bq), (dk, bk), (dv, bv)):
            b += 2.0 ** -8 * (np.abs(x) + b)
        out.append(((dq, dk, dv), (bq, bk, bv)))
    return out


def check_backward(got, want, cq, ck):
    """got: dq, dk, dv tensors; want: reference_backward()."""
    for b, (refs, bounds) in enumerate(want):
        for name, t, cu, ref, bound in zip(("dq", "dk", "dv"), got, (cq, ck, ck), refs, bounds):
            x = n64(t[int(cu[b]):int(cu[b + 1])])
            assert np.isfinite(x).all(), f"sequence {b}: {name} is not finite"
            off = np.abs(x - ref) - bound
            if off.size:
                assert (off <= 0).all(), (f"sequence {b}: {name} is {off.max():.3e} beyond its bound "
                                          f"{bound.flat[off.argmax()]:.3e} at {np.unravel_index(off.argmax(), off.shape)}")


class Cache:
    """A paged cache filled with sequences; every unused row is NaN."""

    def __init__(self, ks, vs, page, seed, spare=3):
        g = gen(seed)
        hk, d = ks[0].shape[1:]
        need = [-(-k.shape[0] // page) for k in ks]
        n = sum(need) + spare
        self.ids = torch.randperm(n, generator=g).tolist()
        self.k = torch.full((n, page, hk, d), math.nan, dtype=torch.bfloat16)
        self.v = self.k.clone()
        self.table = torch.full((len(ks), max(max(need), 1) + 2), -7, dtype=torch.int32)  # never read past the last page
        at = 0
        for b, (k, v) in enumerate(zip(ks, vs)):
            for i in range(need[b]):
                p = self.ids[at]
                at += 1
                self.table[b, i] = p
                part = k[i * page:(i + 1) * page]
                self.k[p, :part.shape[0]] = part
                self.v[p, :part.shape[0]] = v[i * page:(i + 1) * page]
        self.lens = torch.tensor([k.shape[0] for k in ks], dtype=torch.int32)

    def cuda(self):
        for x in ("k", "v", "table", "lens"):
            setattr(self, x, getattr(self, x).cuda())
        return self
