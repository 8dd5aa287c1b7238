"""The block operators' definitions in 64 bits on the CPU, for the tests.

Where a tolerance needs the size of the terms that were added, the same
formula runs with ``mag=True``: every input by its magnitude and every
difference a sum, so that K roundings of 2^-24 each are off by at most
K * 2^-24 times that (first order)."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # one rounding in 32 bits


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def check(name, got, ref, tol):
    """|got - ref| <= tol, element by element, NaN where ref has NaN."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), name
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), name
    ok = ~(nan | inf)
    over = ((got - ref).abs() - tol.expand_as(ref))[ok]
    if over.numel() and not float(over.max()) <= 0.0:
        i = int(over.argmax())
        g, r, t = got[ok][i], ref[ok][i], tol.expand_as(ref)[ok][i]
        raise AssertionError(f"{name}: got {float(g)!r}, expected {float(r)!r} +- {float(t):.3e} "
                             f"({int((over > 0).sum())} of {over.numel()} over)")


# ------------------------------------------------------------ rows by expert
def rows_of(idx, E, capacity_factor=0.0):
    """(offsets, row_entry, entry_row) as lists, entry by entry."""
    N, k = len(idx), len(idx[0]) if len(idx) else 0
    n = N * k
    cap = math.ceil(capacity_factor * n / E) if capacity_factor > 0 else n
    kept, left = [[] for _ in range(E)], [[] for _ in range(E + 1)]
    for i in range(n):
        e = idx[i // k][i % k]
        if not 0 <= e < E:
            left[E].append(i)
        elif len(kept[e]) < cap:
            kept[e].append(i)
        else:
            left[e].append(i)
    offsets, order = [0], []
    for e in range(E):
        order += kept[e]
        offsets.append(len(order))
    row_entry, entry_row = list(order), [None] * n
    for r, i in enumerate(order):
        entry_row[i] = r
    for i in (i for b in left for i in b):
        entry_row[i] = -1 - len(row_entry)
        row_entry.append(-1)
    return offsets, row_entry, entry_row


# ------------------------------------------------------------ norms
def spread_gate(gate, N, H):
    """The gate as [N, H]."""
    if gate is None:
        return torch.ones(N, H, dtype=torch.float64)
    g = gate.double()
    if g.dim() > 1 and g.shape[-1] == 1:
        return g.reshape(N, 1).expand(N, H)
    g = g.reshape(-1, H)
    return g.repeat_interleave(N // g.shape[0], 0) if g.shape[0] else g.expand(N, H)


def norm_bwd(dn, r, w, rstd, mag=False):
    """Gradient of w * r * rstd with respect to r, and dw."""
    if mag:
        dn, r, w = dn.abs(), r.abs(), w.abs()
    rh, a = r * rstd[:, None], dn * w
    t = rh * (a * rh).mean(-1, keepdim=True)
    return rstd[:, None] * (a + t if mag else a - t), (dn * rh).sum(0)


def postnorm_fwd(y, res, w, gate, next_w, scale, eps):
    y, res = y.double(), res.double()
    N, H = y.shape
    g, rstd = spread_gate(gate, N, H), None
    b = y
    if w is not None:
        rstd = 1 / torch.sqrt(y.square().mean(-1) + eps)
        b = y * rstd[:, None] * w.double()
    r = scale * res + g * b
    mag = abs(scale) * res.abs() + (g * b).abs()
    n = next_rstd = None
    if next_w is not None:
        next_rstd = 1 / torch.sqrt(r.square().mean(-1) + eps)
        n = r * next_rstd[:, None] * next_w.double()
    return {"out": r, "rstd": rstd, "n": n, "next_rstd": next_rstd, "mag": mag}


def postnorm_bwd(dout, dn, y, out, w, gate, next_w, rstd, next_rstd, scale, gate_shape=None,
                 mag=False):
    d = (lambda t: t.double().abs()) if mag else (lambda t: t.double())
    y, N, H = d(y), y.shape[0], y.shape[1]
    g = spread_gate(gate, N, H)
    g = g.abs() if mag else g
    dr = torch.zeros(N, H, dtype=torch.float64) if dout is None else d(dout)
    dnext_w = dw = dgate = None
    if next_w is not None:
        t, dnext_w = norm_bwd(dn.double(), out.double(), next_w.double(), next_rstd.double(), mag)
        dr = dr + t
    b, yh, c = dr * g, y, None
    if w is not None:
        c = rstd.double()[:, None]
        yh = y * c
        dw = (dr * g * yh).sum(0)
        b = b * d(w)
        t = yh * (b * yh).mean(-1, keepdim=True)
        dy = c * (b + t if mag else b - t)
    else:
        dy = b
    each = dr * yh * (d(w) if w is not None else 1.0)
    if gate is not None:
        shape = tuple(gate.shape)
        if len(shape) > 1 and shape[-1] == 1:
            dgate = each.sum(-1).reshape(shape)
        else:
            rows = gate.numel() // H
            dgate = (each.reshape(rows, -1, H).sum(1) if rows else each.new_zeros(0, H)).reshape(shape)
    return {"dy": dy, "dresidual": (abs(scale) if mag else scale) * dr, "dw": dw, "dgate": dgate,
            "dnext_w": dnext_w}


# ------------------------------------------------------------ 8 bits
def _e4m3_table():
    """The non-negative finite e4m3 values in order, code by code."""
    t = []
    for code in range(0x7F):
        e, m = code >> 3, code & 7
        t.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(t, dtype=torch.float64)


E4M3 = _e4m3_table()


def to_e4m3(v):
    """Codes (int64) of the e4m3 values nearest to v (|v| <= 448), ties to the even code."""
    a = v.abs()
    hi = torch.searchsorted(E4M3, a).clamp(max=E4M3.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return pick + 128 * torch.signbit(v).long()


def act8(x):
    """(codes [R, C], scale bytes [R, ceil(C / 32)], values) of x; NaN's code is 0x7f here."""
    x = x.double()
    R, C = x.shape
    G = -(-C // 32)
    fine = torch.isfinite(x)
    a = torch.nn.functional.pad(torch.where(fine, x.abs(), torch.zeros_like(x)), (0, G * 32 - C))
    a = a.reshape(R, G, 32).amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1): 448 2^s = 0.875 2^(s + 9)
    s = torch.where(a > 0, (e - 9 + (m > 0.875)).clamp(min=-127), torch.full_like(e, -127)).long()
    at = s.repeat_interleave(32, 1)[:, :C]
    scale = torch.exp2(at.double())
    v = torch.where(fine, x / scale, torch.zeros_like(x))
    codes = to_e4m3(v)
    codes = torch.where(fine, codes, torch.full_like(codes, 0x7F))
    return codes, (s + 127).to(torch.uint8), from_act8(codes, (s + 127).to(torch.uint8))


def from_act8(codes, scale):
    codes, C = codes.long(), codes.shape[1]
    low = codes & 0x7F
    v = torch.where(low == 0x7F, torch.full_like(low, 1).double() * math.nan,
                    E4M3[low.clamp(max=0x7E)])
    v = torch.where(codes >= 128, -v, v)
    return v * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)[:, :C]


def silu_terms(g, u, dh=None):
    """h = silu(g) u and with dh also (dg, du), each with its tolerance in 32 bits.

    The kernel's sigmoid is 1 / (1 + 2^t), t = -g log2(e) rounded twice (the
    constant, the product): t is off by 2 |t| 2^-24, so 2^t by 2 |g| 2^-24
    relative, plus one unit (2^-23) of each of v_exp_f32 and v_rcp_f32 and the
    sum's rounding: K = 2 |g| + 5 in units of 2^-24, and four more roundings
    for the products.  In dg, 1 - s is off by K s 2^-24 absolutely.  Where the
    sigmoid falls below the smallest normal number it may be taken as 0."""
    K = 2 * g.abs() + 10
    tiny = 2.0 ** -125
    e = torch.exp(-g)
    s = 1 / (1 + e)
    one_s = torch.where(torch.isinf(e), torch.ones_like(e), e / (1 + e))
    h = g * s * u
    out = [(h, K * U32 * h.abs() + tiny * (1 + g.abs()) * (1 + u.abs()))]
    if dh is not None:
        dg = dh * u * s * (1 + g * one_s)
        mag = (dh * u).abs() * s * (1 + g.abs() * one_s + g.abs() * s)
        out.append((dg, K * U32 * mag + tiny * (1 + g.abs()) * (1 + (dh * u).abs())))
        du = dh * g * s
        out.append((du, K * U32 * du.abs() + tiny * (1 + g.abs()) * (1 + dh.abs())))
    return out
