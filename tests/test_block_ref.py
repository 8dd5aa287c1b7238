"""The 64-bit definitions the block operators are tested against, themselves
checked: gradients against differences, the 8-bit grid against torch's."""
import pytest
import torch

import block_ref as R


def test_rows_small():
    offsets, row_entry, entry_row = R.rows_of([[1, 0], [1, -1], [1, 1], [5, 0]], 2, 0.5)
    # cap = ceil(0.5 * 8 / 2) = 2; expert 0: entries 1, 7; expert 1: 0, 2 (4, 5 over); none: 3, 6
    assert offsets == [0, 2, 4]
    assert row_entry == [1, 7, 0, 2, -1, -1, -1, -1]
    assert entry_row == [2, 0, 3, -7, -5, -6, -8, 1]


@pytest.mark.parametrize("norm,gate_shape,nxt", [(True, (3, 8), True), (True, (6, 1), False),
                                                 (False, (8,), True), (True, None, True)])
def test_postnorm_gradient_by_differences(norm, gate_shape, nxt):
    g = torch.Generator().manual_seed(3)
    N, H, eps, scale = 6, 8, 1e-3, 0.75
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    t = {"y": rnd(N, H), "res": rnd(N, H), "w": rnd(H) if norm else None,
         "gate": rnd(*gate_shape) if gate_shape else None, "next_w": rnd(H) if nxt else None}
    dout, dn = rnd(N, H), rnd(N, H)

    def loss():
        f = R.postnorm_fwd(t["y"], t["res"], t["w"], t["gate"], t["next_w"], scale, eps)
        return float((f["out"] * dout).sum() + ((f["n"] * dn).sum() if nxt else 0.0))

    f = R.postnorm_fwd(t["y"], t["res"], t["w"], t["gate"], t["next_w"], scale, eps)
    b = R.postnorm_bwd(dout, dn, t["y"], f["out"], t["w"], t["gate"], t["next_w"], f["rstd"],
                       f["next_rstd"], scale)
    for name, grad in (("y", b["dy"]), ("res", b["dresidual"]), ("w", b["dw"]),
                       ("gate", b["dgate"]), ("next_w", b["dnext_w"])):
        if t[name] is None:
            continue
        flat = t[name].view(-1)
        for i in range(flat.numel()):
            keep, h = float(flat[i]), 1e-5
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            # central differences: error of order h^2 times third derivatives (tens here)
            assert abs((up - down) / (2 * h) - float(grad.reshape(-1)[i])) < 1e-6, (name, i)


def test_silu_gradient_by_differences():
    g = torch.linspace(-12, 12, 97, dtype=torch.float64)
    u, dh, h = g.flip(0) * 0.3 + 1, g * 0 + 0.7, 1e-6
    _, (dg, _), (du, _) = R.silu_terms(g, u, dh)
    f = lambda a, b: R.silu_terms(a, b)[0][0] * dh
    assert float(((f(g + h, u) - f(g - h, u)) / (2 * h) - dg).abs().max()) < 1e-8
    assert float(((f(g, u + h) - f(g, u - h)) / (2 * h) - du).abs().max()) < 1e-8


def test_e4m3_grid_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double()
    mine = R.from_act8(codes[None].expand(1, 256), torch.full((1, 8), 127, dtype=torch.uint8))[0]
    assert torch.equal(torch.isnan(t), torch.isnan(mine))
    ok = ~torch.isnan(t)
    assert torch.equal(t[ok], mine[ok])
    v = torch.cat([torch.linspace(-448, 448, 4001), torch.linspace(-0.04, 0.04, 4001)])
    assert torch.equal(R.to_e4m3(v.double()), v.to(torch.float8_e4m3fn).view(torch.uint8).long())


def test_act8_scales():
    x = torch.zeros(6, 40)
    x[1, 0], x[1, 39] = 448.0, 449.0
    x[2, 3], x[2, 4] = -449.0, float("inf")
    x[3, 0] = 2.0 ** -140
    x[4, 5], x[4, 6] = float("nan"), 3.0e38
    codes, scale, v = R.act8(x)
    assert scale.tolist()[:4] == [[0, 0], [127, 128], [128, 0], [0, 0]]
    assert float(v[1, 0]) == 448.0 and float(v[1, 39]) == 448.0  # 449 / 2 = 224.5 -> 224
    assert torch.isnan(v[2, 4]) and float(v[2, 3]) == -448.0
    assert torch.isnan(v[4, 5]) and abs(float(v[4, 6]) / 3.0e38 - 1) <= 2.0 ** -4


def test_act8_error_bound():
    """A kept value is within max(2^-4 |x|, 2^-10 2^e) of x: relative where e4m3's numbers are
    normal, absolute below, where 2^-4 |x| alone does not hold and small elements become 0."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(64, 96, generator=g, dtype=torch.float64).float().double()
    x = x * torch.exp2(-torch.randint(0, 30, x.shape, generator=g).double())  # within one group
    x[5] *= 2.0 ** -100
    codes, scale, v = R.act8(x)
    unit = torch.exp2(scale.double() - 127).repeat_interleave(32, 1)
    err = (v - x).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * unit)).all())
    assert bool((err > 2.0 ** -4 * x.abs()).any())
    assert torch.equal(v == 0, x.abs() <= 2.0 ** -10 * unit)
    group = x.abs().reshape(64, 3, 32).amax(-1).repeat_interleave(32, 1)
    lost = v == 0
    assert bool(lost.any()) and bool((x.abs()[lost] <= 2.0 ** -17 * group[lost]).all())
    assert bool((v[x.abs() > 2.0 ** -17 * group] != 0).all())
