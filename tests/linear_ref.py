"""The products of rows by expert and the 4-bit format in 64 bits on the CPU, for the tests.

A sum of L products in 32 bits, added in any order, is off by at most L * 2^-24 of the sum of the
products' magnitudes (first order; the products themselves are exact or off by half a step each:
counted as one more), whatever the order."""
from __future__ import annotations

import math

import torch

from block_ref import U32, half_step

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def to_e2m1(v):
    """Codes (int64) of the e2m1 values nearest to v (|v| <= 6), ties to the even code."""
    a = v.abs()
    hi = torch.searchsorted(E2M1, a).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return pick + 8 * torch.signbit(v).long()


def mx4(x):
    """(q bytes [..., C / 2], scale bytes [..., ceil(C / 32)]) of x [..., C]."""
    x = x.double()
    C = x.shape[-1]
    G = -(-C // 32)
    pad = torch.nn.functional.pad(x, (0, G * 32 - C)).reshape(*x.shape[:-1], G, 32)
    bad = ~torch.isfinite(pad).all(-1)
    a = torch.where(bad[..., None], torch.zeros_like(pad), pad).abs().amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1): 6 2^s = 0.75 2^(s + 3)
    s = torch.where(a > 0, (e - 3 + (m > 0.75)).clamp(min=-127), torch.full_like(e, -127)).long()
    v = torch.where(bad[..., None], torch.zeros_like(pad), pad) / torch.exp2(s.double())[..., None]
    codes = to_e2m1(v)
    codes = torch.where(bad[..., None], torch.zeros_like(codes), codes)
    codes = codes.reshape(*x.shape[:-1], G * 32)[..., :C]
    scale = torch.where(bad, torch.full_like(s, 255), s + 127)
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8), scale.to(torch.uint8)


def from_mx4(q, scale):
    codes = torch.stack([q.long() % 16, q.long() // 16], -1).flatten(-2)
    v = E2M1[codes % 8] * (1 - 2 * (codes // 8)).double()
    s = torch.exp2(scale.double() - 127)
    s = torch.where(scale == 255, torch.full_like(s, math.nan), s)
    return v * s.repeat_interleave(32, -1)[..., :codes.shape[-1]]


def grouped(x, mats, sizes, R=None):
    """y[r] = mats[e] x[r] for the groups of rows, zeros behind them."""
    y = torch.zeros(x.shape[0] if R is None else R, mats.shape[1], dtype=torch.float64)
    b = 0
    for e, n in enumerate(sizes):
        y[b:b + n] = x[b:b + n].double() @ mats[e].double().T
        b += n
    return y


def grouped_dw(dy, x, sizes):
    dw, b = torch.zeros(len(sizes), dy.shape[1], x.shape[1], dtype=torch.float64), 0
    for e, n in enumerate(sizes):
        dw[e] = dy[b:b + n].double().T @ x[b:b + n].double()
        b += n
    return dw


def tol(ref, mag, terms, dtype):
    """``terms`` products added in 32 bits, the result rounded to dtype (subnormals of fp32 may be
    taken as 0)."""
    return half_step(dtype) * ref.abs() + (terms + 1) * U32 * mag * (1 + half_step(dtype)) + 2.0 ** -126
