"""Products of rows by expert with their gradients, and matrices in 4 bits, on the GPU against their
64-bit definitions (linear_ref).

Tolerances count roundings: half a step of the output's type, and one of 2^-24 for each product of a
sum, of the sum of the products' magnitudes."""
import math

import pytest
import torch

import block_ref as BR
import linear_ref as R
from gpu_util import announce, torch_dev

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BITS = {torch.bfloat16: torch.int16, torch.float32: torch.int32}


@pytest.fixture(scope="module")
def env():
    torch_, dev = torch_dev()
    import top_moe_layer_amd as tm

    tm.lib()
    return dev, tm


def rnd(seed, *shape, dt=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dt)


def offsets(sizes):
    return torch.tensor([0] + torch.tensor(sizes, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int32)


def same(a, b):
    a, b = a.detach().cpu(), b.detach().cpu()
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(
        a.contiguous().view(BITS.get(a.dtype, a.dtype)), b.contiguous().view(BITS.get(b.dtype, b.dtype)))


def pitched(t, dev, more=8):
    """t [R, C] on the GPU as a view of rows ``more`` elements longer, NaN between them."""
    big = torch.full((t.shape[0], t.shape[1] + more), math.nan, dtype=t.dtype, device=dev)
    big[:, :t.shape[1]] = t.to(dev)
    return big[:, :t.shape[1]]


# rows of each expert, rows of none behind them, K, O: ragged groups, empty experts, sizes that end
# inside every tile, one element past them, and of each kernel's own range
SMALL = [
    ([0], 0, 8, 8), ([1], 0, 8, 8), ([1], 0, 2048, 264), ([0, 0, 1], 3, 16, 24),
    ([3, 0, 17], 2, 64, 40), ([16, 15, 1, 0], 0, 136, 1000), ([40] * 3, 5, 96, 72),
    ([130, 0, 65, 257, 5], 70, 72, 136), ([64, 128], 0, 128, 256), ([63, 129, 1], 1, 200, 264),
    ([2] * 256, 7, 32, 16), ([1] * 70 + [0] * 100 + [9] * 3, 0, 40, 48),
]
LARGE = [  # 128 x 256 and 256 x 256 tiles, NT by O, NN by K; sums long enough for parts
    ([349, 351], 5, 72, 5960), ([600, 705], 9, 40, 6008), ([349, 351], 5, 5960, 72),
    ([600, 705], 0, 6008, 40), ([257], 0, 64, 35848),
    ([900, 40, 100], 60, 264, 520), ([2400, 0, 260, 300, 280, 310, 250, 1000], 100, 136, 72),
    ([300] * 15 + [1700], 0, 24, 40), ([20], 3, 64, 6464), ([5, 30, 0], 1, 1032, 1160),
    ([1500, 1700], 40, 264, 6152), ([1500, 1700], 0, 6152, 264),  # several tiles a block
    ([1433, 621], 5, 2568, 2440), ([349, 251], 5, 2568, 2440),  # tiles of 256 x 256 and 128 x 256 for dw
    ([5000], 9, 136, 264), ([4100, 0, 700], 20, 72, 40),  # parts that fill the CUs
]


def linear_case(env, sizes, extra, K, O, dt, pitch):
    dev, tm = env
    d, E, n = DT[dt], len(sizes), sum(sizes)
    Rn = n + extra
    x, dy = rnd(1, Rn, K, dt=d), rnd(2, Rn, O, dt=d)
    w = rnd(3, E, O, K, dt=d, scale=K ** -0.5)
    x[n:] = math.nan  # rows of no expert are not read
    dy[n:] = math.inf
    on = (lambda t: pitched(t, dev)) if pitch else (lambda t: t.to(dev))
    off = offsets(sizes).to(dev)
    xd, dyd, wd = on(x), on(dy), w.to(dev)
    y = tm.moe_linear_fwd(xd, wd, off)
    g = tm.moe_linear_bwd(dyd, xd, wd, off)
    torch.cuda.synchronize()
    wt = w.transpose(1, 2)
    ref = R.grouped(x, w, sizes)
    BR.check("y", y, ref, R.tol(ref, R.grouped(x.abs(), w.abs(), sizes), K, d))
    ref = R.grouped(dy, wt, sizes)
    BR.check("dx", g.dx, ref, R.tol(ref, R.grouped(dy.abs(), wt.abs(), sizes), O, d))
    ref = R.grouped_dw(dy, x, sizes)
    BR.check("dw", g.dw, ref, R.tol(ref, R.grouped_dw(dy.abs(), x.abs(), sizes), max(sizes), d))
    # every call, and either gradient alone, gives the same bits
    assert same(y, tm.moe_linear_fwd(xd, wd, off))
    assert same(g.dx, tm.moe_linear_bwd(dyd, None, wd, off, need_dw=False).dx)
    assert same(g.dw, tm.moe_linear_bwd(dyd, xd, wd, off, need_dx=False).dw)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes,extra,K,O", SMALL)
def test_linear(env, sizes, extra, K, O, dt):
    announce(f"linear {len(sizes)} experts, {sum(sizes)} + {extra} rows, {K} -> {O} {dt}")
    linear_case(env, sizes, extra, K, O, dt, pitch=len(sizes) % 2 == 1)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes,extra,K,O", LARGE)
def test_linear_large_tiles(env, sizes, extra, K, O, dt):
    announce(f"linear {len(sizes)} experts, {sum(sizes)} + {extra} rows, {K} -> {O} {dt}")
    linear_case(env, sizes, extra, K, O, dt, pitch=len(sizes) % 2 == 1)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_linear_one_matrix(env, dt):
    """Without offsets, [O, K] and [1, O, K]: all rows, nothing behind them."""
    dev, tm = env
    d = DT[dt]
    for n, K, O in ((1, 64, 72), (50, 136, 40), (300, 72, 264), (2600, 72, 40)):
        x, w, dy = rnd(1, n, K, dt=d), rnd(2, O, K, dt=d), rnd(3, n, O, dt=d)
        D = [t.to(dev) for t in (x, w, dy)]
        y = tm.moe_linear_fwd(D[0], D[1])
        assert same(y, tm.moe_linear_fwd(D[0], D[1][None]))
        assert same(y, tm.moe_linear_fwd(D[0], D[1][None], offsets([n]).to(dev)))
        ref = x.double() @ w.double().T
        BR.check("y", y, ref, R.tol(ref, x.double().abs() @ w.double().abs().T, K, d))
        g = tm.moe_linear_bwd(D[2], D[0], D[1])
        assert g.dw.shape == w.shape
        ref = dy.double().T @ x.double()
        BR.check("dw", g.dw, ref, R.tol(ref, dy.double().abs().T @ x.double().abs(), n, d))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_values_that_are_not_finite_stay_in_their_row_and_expert(env, dt):
    dev, tm = env
    d, sizes, K, O = DT[dt], [20, 70, 0, 33], 104, 136
    off = offsets(sizes).to(dev)
    x, w, dy = rnd(1, 123, K, dt=d), rnd(2, 4, O, K, dt=d), rnd(3, 123, O, dt=d)
    clean = tm.moe_linear_fwd(x.to(dev), w.to(dev), off)
    cg = tm.moe_linear_bwd(dy.to(dev), x.to(dev), w.to(dev), off)
    x2, dy2 = x.clone(), dy.clone()
    x2[25, 7], dy2[100, 9] = math.nan, math.inf
    y = tm.moe_linear_fwd(x2.to(dev), w.to(dev), off)
    g = tm.moe_linear_bwd(dy2.to(dev), x2.to(dev), w.to(dev), off)
    torch.cuda.synchronize()
    rows = torch.arange(123)
    assert torch.isnan(y[25]).all() and same(y[rows != 25], clean[rows != 25])
    assert not torch.isfinite(g.dx[100]).any() and same(g.dx[rows != 100], cg.dx[rows != 100])
    assert torch.isnan(g.dw[1, :, 7]).all() and same(g.dw[[0, 2]], cg.dw[[0, 2]])
    cols = torch.arange(K) != 7
    assert same(g.dw[1][:, cols], cg.dw[1][:, cols])
    outs = torch.arange(O) != 9
    assert not torch.isfinite(g.dw[3, 9]).any() and same(g.dw[3][outs], cg.dw[3][outs])


def test_offsets_out_of_range(env):
    """Offsets that decrease or lie outside [0, R] give other rows, but write nothing outside."""
    dev, tm = env
    d, Rn, K, O = torch.bfloat16, 90, 64, 72
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((Rn, K), (5, O, K), (Rn, O))))
    for off in ([0, 30, 20, 60, 50, 90], [5, 10, 2 ** 31 - 1, 40, -7, 90], [-2 ** 31] * 6, [90] * 6):
        o = torch.tensor(off, dtype=torch.int32, device=dev)
        big = torch.full((Rn + 512, O), 7.0, dtype=d, device=dev)
        tm.moe_linear_fwd(x, w, o, y=big[256:256 + Rn])
        bdx = torch.full((Rn + 512, K), 7.0, dtype=d, device=dev)
        bdw = torch.full((15, O, K), 7.0, dtype=d, device=dev)
        tm.moe_linear_bwd(dy, x, w, o, dx=bdx[256:256 + Rn], dw=bdw[5:10])
        torch.cuda.synchronize()
        for b in (big, bdx):
            assert bool((b[:256] == 7).all()) and bool((b[256 + Rn:] == 7).all())
        assert bool((bdw[:5] == 7).all()) and bool((bdw[10:] == 7).all())


def test_offsets_out_of_range_in_parts(env):
    """The same where dw is summed in parts: each expert claims all rows."""
    dev, tm = env
    d, E, Rn, K, O = torch.bfloat16, 8, 2400, 72, 136
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((Rn, K), (E, O, K), (Rn, O))))
    o = torch.tensor([0, Rn] * 4 + [0], dtype=torch.int32, device=dev)
    need = tm.moe_linear_bwd_workspace_bytes(Rn, K, O, E)
    assert need > 256
    ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device=dev)
    tm.moe_linear_bwd(dy, x, w, o, workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 7).all())


def test_gradients_are_differences(env):
    """y is linear in x and in w: its change along a direction is the gradient's product with it."""
    dev, tm = env
    sizes, K, O = [7, 0, 60, 13], 40, 56
    off = offsets(sizes).to(dev)
    x, w, dy, vx, vw = (rnd(i, *s).to(dev) for i, s in enumerate(
        ((80, K), (4, O, K), (80, O), (80, K), (4, O, K))))
    g = tm.moe_linear_bwd(dy, x, w, off)
    f = lambda a, b: tm.moe_linear_fwd(a, b, off).double()
    h = 0.5
    for grad, v, plus, minus in ((g.dx, vx, f(x + h * vx, w), f(x - h * vx, w)),
                                 (g.dw, vw, f(x, w + h * vw), f(x, w - h * vw))):
        # differences of sums of K terms of about 2^2 each in 32 bits, 80 * 56 of them
        want = float(((plus - minus) / (2 * h) * dy.double()).sum())
        got = float((grad.double() * v.double()).sum())
        mag = float((f(x.abs(), w.abs()) * dy.abs().double()).sum())
        assert abs(got - want) <= (K + O + 80) * 2.0 ** -22 * mag


# ------------------------------------------------------------ 4 bits
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("Rn,C", [(1, 8), (1, 32), (3, 40), (7, 64), (65, 96), (33, 1000), (5, 8200)])
def test_mx4_round_trip(env, Rn, C, dt):
    dev, tm = env
    announce(f"mx4 {Rn} x {C} {dt}")
    d = DT[dt]
    g = torch.Generator().manual_seed(Rn + C)
    x = rnd(Rn, Rn, C) * torch.exp2(torch.randint(-40, 40, (Rn, C), generator=g).float() *
                                    (torch.rand(Rn, 1, generator=g) < 0.5))
    x[torch.rand(Rn, C, generator=g) < 0.05] = 0.0
    x = x.to(d)
    if Rn > 4:
        x[1, C // 2], x[2, 0], x[3, C - 1] = math.nan, math.inf, -math.inf
        x[4, :32] = 0.0
    for on in (x.to(dev), pitched(x, dev, 24)):
        p = tm.mx4_pack(on)
        torch.cuda.synchronize()
        q, s = R.mx4(x)
        assert torch.equal(p.scale.cpu(), s)
        assert torch.equal(p.q.cpu(), q)
    for out in DT.values():
        want = R.from_mx4(q, s)
        got = tm.mx4_unpack(p, dtype=out)
        # e2m1 and a power of two: exact in either type
        BR.check("values", got, want.to(out).double(), torch.zeros_like(want))
        into = torch.full((Rn, C + 16), 5.0, dtype=out, device=dev)
        tm.mx4_unpack(p, x=into[:, :C])
        torch.cuda.synchronize()
        assert same(into[:, :C].contiguous(), got) and bool((into[:, C:] == 5).all())


def test_mx4_every_bf16_value(env):
    """Every finite bf16 value as its group's largest, and beside one: ties, subnormals, the range's ends."""
    dev, tm = env
    v = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    for top in (0.0, 1.0, 6.0, 3e38, 2.0 ** -130):
        x = torch.zeros(v.numel(), 8, dtype=torch.bfloat16)
        x[:, 0], x[:, 5] = v, top
        for t in (x, x.float()):
            p = tm.mx4_pack(t.to(dev))
            torch.cuda.synchronize()
            q, s = R.mx4(x)
            assert torch.equal(p.scale.cpu(), s) and torch.equal(p.q.cpu(), q), top
            want = R.from_mx4(q, s)
            BR.check("fp32", tm.mx4_unpack(p, dtype=torch.float32), want.float().double(),
                     torch.zeros_like(want))


def test_mx4_every_code(env):
    dev, tm = env
    scale = torch.arange(256, dtype=torch.uint8)[:, None]
    q = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).clone()
    q[:, 1:] = (q[:, 1:] + torch.arange(15, dtype=torch.uint8) * 17) & 255
    for out in DT.values():
        got = tm.mx4_unpack(tm.Mx4(q.to(dev), scale.to(dev)), dtype=out)
        torch.cuda.synchronize()
        want = R.from_mx4(q, scale)
        BR.check("values", got, want.to(out).double(), torch.zeros_like(want))


def test_mx4_leading_dimensions(env):
    dev, tm = env
    w = rnd(1, 3, 5, 72).to(dev)
    p = tm.mx4_pack(w)
    assert p.q.shape == (3, 5, 36) and p.scale.shape == (3, 5, 3)
    flat = tm.mx4_pack(w.reshape(15, 72))
    assert torch.equal(p.q.reshape(15, 36), flat.q) and torch.equal(p.scale.reshape(15, 3), flat.scale)
    assert same(tm.mx4_unpack(p, dtype=torch.float32).reshape(15, 72),
                tm.mx4_unpack(flat, dtype=torch.float32))
    e = tm.mx4_pack(torch.empty(0, 64, device=dev))
    assert e.q.shape == (0, 32) and tm.mx4_unpack(e).shape == (0, 64)


MX = [  # K in whole groups, tails of one to three groups behind slices of 4 and 8
    ([0], 0, 32, 8), ([1], 0, 32, 8), ([1], 0, 2048, 264), ([0, 3, 0, 17], 2, 96, 40),
    ([16, 15, 1], 3, 160, 1000), ([40] * 3, 5, 224, 72), ([130, 0, 65, 257, 5], 70, 352, 136),
    ([64, 128], 0, 128, 256), ([2] * 200, 7, 32, 16), ([700], 0, 64, 12808), ([300] * 4, 9, 416, 2568),
    ([30], 0, 1056, 512), ([700], 1, 96, 17608), ([1500, 1700], 0, 288, 6152),
    # scales in whole words, and of each shape of tiles
    ([130, 0, 65, 257, 5], 70, 384, 136), ([1500, 1700], 0, 256, 6152), ([600, 705], 9, 128, 6008),
    ([1400, 1300], 30, 1152, 3592), ([300] * 4, 9, 1024, 4104),
]
# 8-bit rows with y in bf16: of eight products each may lose what lies 2^-13 and less of the largest
WINDOW = 8 * 2.0 ** -13


@pytest.mark.parametrize("kind", ["bf16", "fp32", "act8>bf16", "act8>fp32", "mx4>bf16", "mx4>fp32"])
@pytest.mark.parametrize("sizes,extra,K,O", MX)
def test_mx4_linear(env, sizes, extra, K, O, kind):
    dev, tm = env
    announce(f"mx4 linear {len(sizes)} experts, {sum(sizes)} + {extra} rows, {K} -> {O} {kind}")
    rows, _, out = kind.partition(">")
    out = DT[out or rows]
    n = sum(sizes)
    x = rnd(1, n + extra, K, dt=DT.get(rows, torch.float32))
    w = rnd(2, len(sizes), O, K, scale=K ** -0.5)
    w = w * torch.exp2(torch.randint(-8, 8, (len(sizes), O, 1), generator=torch.Generator().manual_seed(4)).float())
    q, s = R.mx4(w)
    W, off = tm.Mx4(q.to(dev), s.to(dev)), offsets(sizes).to(dev)
    wv = R.from_mx4(q, s)
    if rows in DT:
        x[n:] = math.nan
        arg, xv = pitched(x, dev), x
    elif rows == "act8":
        arg = tm.act8_pack(x.to(dev))
        codes, scale, xv = BR.act8(x)
        arg.scale[n:] = 255  # NaN in rows of no expert
    else:
        arg = tm.mx4_pack(x.to(dev))
        xv = R.from_mx4(*R.mx4(x))
        arg.scale[n:] = 255
    y = tm.mx4_linear_fwd(arg, W, off, dtype=out)
    torch.cuda.synchronize()
    ref, mag = R.grouped(xv, wv, sizes), R.grouped(xv.double().abs(), wv.abs(), sizes)
    tol = R.tol(ref, mag, K, out) + (WINDOW * mag if kind == "act8>bf16" else 0)
    BR.check("y", y, ref, tol)
    assert same(y, tm.mx4_linear_fwd(arg, W, off, dtype=out))
    if rows in DT:
        dy = rnd(3, n + extra, O, dt=out)
        dy[n:] = math.nan
        dx = tm.mx4_linear_bwd(pitched(dy, dev), W, off)
        torch.cuda.synchronize()
        wt = wv.transpose(1, 2)
        ref = R.grouped(dy, wt, sizes)
        BR.check("dx", dx, ref, R.tol(ref, R.grouped(dy.double().abs(), wt.abs(), sizes), O, out))


@pytest.mark.parametrize("K", [160, 256])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_mx4_linear_scales(env, n, K):
    """The scales' whole range: matrices of 2^-127 and up, a scale of NaN in one column and in one
    row, rows whose scales meet them."""
    dev, tm = env
    O = 72
    g = torch.Generator().manual_seed(n)
    q = torch.randint(0, 256, (O, K // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    s = (torch.arange(O * (K // 32)) * 7 % 250).reshape(O, K // 32).to(torch.uint8)
    s[11, 3] = 255
    wv = R.from_mx4(q, s)
    W = tm.Mx4(q.to(dev), s.to(dev))
    x = rnd(2, n, K)
    p = tm.mx4_pack(x.to(dev))
    if n > 1:
        p.scale[n // 2, K // 32 - 1] = 255
    xv = R.from_mx4(p.q.cpu(), p.scale.cpu())
    for arg, v, d in ((x.to(dev), x, torch.float32), (x.bfloat16().to(dev), x.bfloat16(), torch.bfloat16),
                      (p, xv, torch.float32), (p, xv, torch.bfloat16)):
        y = tm.mx4_linear_fwd(arg, W, dtype=d)
        torch.cuda.synchronize()
        ref, mag = v.double() @ wv.T, v.double().abs() @ wv.abs().T
        fine = mag.isnan() | (mag < 2.0 ** 127)
        assert bool(fine.any()) and torch.equal(y.cpu().isnan(), ref.isnan())
        BR.check("y", torch.where(fine, y.cpu().double(), 0.0), torch.where(fine, ref, 0.0),
                 torch.where(fine, R.tol(ref, mag, K, d), torch.tensor(0.0, dtype=torch.float64)))


@pytest.mark.parametrize("n", [3, 70, 700])
def test_mx4_linear_scales_at_any_address(env, n):
    """Scales that begin at odd addresses, of rows and of matrices, change no bit."""
    dev, tm = env
    K, O = 256, 6152
    p, W = tm.mx4_pack(rnd(1, n, K).to(dev)), tm.mx4_pack(rnd(2, O, K).to(dev))
    a8 = tm.act8_pack(rnd(1, n, K).to(dev))

    def moved(t, by):
        big = torch.full((t.numel() + 64,), 255, dtype=torch.uint8, device=dev)
        big[by:by + t.numel()] = t.reshape(-1)
        return big[by:by + t.numel()].view(t.shape)

    for x in (p, a8, rnd(1, n, K).to(dev), rnd(1, n, K).to(dev).bfloat16()):
        for d in (torch.bfloat16, torch.float32):
            if isinstance(x, torch.Tensor) and x.dtype != d:
                continue
            want = tm.mx4_linear_fwd(x, W, dtype=d)
            for by in (1, 2, 4):
                got = tm.mx4_linear_fwd(x, tm.Mx4(W.q, moved(W.scale, by)), dtype=d)
                assert same(got, want)
                if not isinstance(x, torch.Tensor):
                    assert same(tm.mx4_linear_fwd(x._replace(scale=moved(x.scale, by)), W, dtype=d), want)


@pytest.mark.parametrize("n", [2, 100])
def test_mx4_linear_fp32_rows_of_every_kind(env, n):
    """fp32 rows as they are: 24 bits, next to the range's ends, infinities, NaN; each in its own row."""
    dev, tm = env
    K, O = 64, 40
    w = rnd(1, O, K)
    q, s = R.mx4(w)
    wv = R.from_mx4(q, s)
    for v in (1 + 2.0 ** -23, 16777215.0, 3.4e38, -2.0 ** -126, 1.5 * 2.0 ** -120, math.inf, -math.inf, math.nan):
        x = torch.zeros(n, K)
        x[1, 5] = v
        x[0] = 1.0
        y = tm.mx4_linear_fwd(x.to(dev), tm.Mx4(q.to(dev), s.to(dev)))
        torch.cuda.synchronize()
        ref, mag = x.double() @ wv.T, x.double().abs() @ wv.abs().T
        big = mag > 3.4e38  # past fp32's range
        ref32 = torch.where(big & ref.isfinite(), torch.sign(ref) * math.inf, ref)
        BR.check("y", y, ref32, torch.where(mag.isfinite(), R.tol(ref, mag, K, torch.float32), torch.zeros_like(mag)))


# ------------------------------------------------------------ in use
def leaves(*ts):
    return [t.clone().requires_grad_() for t in ts]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_functions_are_their_entry_points(env, dt):
    dev, tm = env
    d, sizes, K, O = DT[dt], [33, 0, 70, 9], 96, 72
    off = offsets(sizes).to(dev)
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((120, K), (4, O, K), (120, O))))
    a, b = leaves(x, w)
    y = tm.moe_linear(a, b, off)
    assert same(y, tm.moe_linear_fwd(x, w, off))
    y.backward(dy)
    g = tm.moe_linear_bwd(dy, x, w, off)
    assert same(a.grad, g.dx) and same(b.grad, g.dw)
    a, = leaves(x)
    tm.moe_linear(a, w, off).backward(dy)
    assert same(a.grad, g.dx)
    b, = leaves(w)
    tm.moe_linear(x, b, off).backward(dy)
    assert same(b.grad, g.dw)
    # an expanded gradient
    a, b = leaves(x, w)
    tm.moe_linear(a, b, off).sum().backward()
    assert same(a.grad, tm.moe_linear_bwd(torch.ones_like(dy), x, w, off).dx)
    p = tm.mx4_pack(w)
    a, = leaves(x)
    y = tm.mx4_linear(a, p, off)
    assert same(y, tm.mx4_linear_fwd(x, p, off))
    y.backward(dy)
    assert same(a.grad, tm.mx4_linear_bwd(dy, p, off))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_moe_of_own_experts(env, dt, four):
    """Dispatch, gate and up projection, SwiGLU, down projection, combine: the framework's own MoE of
    the same weights, and its gradients by the formulas."""
    dev, tm = env
    d, N, H, I, E, k = DT[dt], 50, 64, 128, 5, 2  # (the framework's own takes multiples of 64)
    x, Wr = rnd(1, N, H, dt=d), rnd(2, E, H, scale=H ** -0.5)
    Wgu, Wd = rnd(3, E, 2 * I, H, dt=d, scale=H ** -0.5), rnd(4, E, H, I, dt=d, scale=I ** -0.5)
    if four:
        pgu, pd = tm.mx4_pack(Wgu.to(dev)), tm.mx4_pack(Wd.to(dev))
        Wgu, Wd = (tm.mx4_unpack(p, dtype=d).cpu() for p in (pgu, pd))
    D = [t.to(dev) for t in (x, Wr, Wgu, Wd)]
    out = tm.moe_ffn_fwd(D[0], D[1], D[2][:, :I].contiguous(), D[2][:, I:].contiguous(), D[3], k, 0.0)
    xl, gul, dl = leaves(D[0], D[2], D[3])
    r = tm.moe_dispatch(xl, out.topk_idx, E)
    gu = tm.mx4_linear(r.xs, pgu, r.expert_offsets) if four else tm.moe_linear(r.xs, gul, r.expert_offsets)
    h = tm.swiglu_act8(gu)
    ys = tm.mx4_linear(h, pd, r.expert_offsets) if four else tm.moe_linear(h, dl, r.expert_offsets)
    y = tm.moe_combine(ys, r.entry_row, out.alpha)
    ref, got = out.y.double(), y.detach().double()
    # both round gu or h and ys to the type on the way: a few half steps of the largest values
    few = 16 * R.half_step(d) * float(ref.abs().max()) + (1e-5 if dt == "fp32" else 0)
    assert float((got - ref).abs().max()) <= few
    dy = rnd(5, N, H, dt=d).to(dev)
    y.backward(dy)
    # the formulas, in 64 bits
    X, GU, DN, al, idx, dY = (t.detach().double().cpu() for t in (D[0], D[2], D[3], out.alpha, out.topk_idx, dy))
    dX = torch.zeros(N, H, dtype=torch.float64)
    dGU, dDN = torch.zeros(E, 2 * I, H, dtype=torch.float64), torch.zeros(E, H, I, dtype=torch.float64)
    for t in range(N):
        for j in range(k):
            e = int(idx[t, j])
            v = GU[e] @ X[t]
            s = torch.sigmoid(v[:I])
            hh = v[:I] * s * v[I:]
            do = al[t, j] * dY[t]
            dh = DN[e].T @ do
            dv = torch.cat([dh * v[I:] * s * (1 + v[:I] * (1 - s)), dh * v[:I] * s])
            dX[t] += GU[e].T @ dv
            dGU[e] += torch.outer(dv, X[t])
            dDN[e] += torch.outer(do, hh)
    # g and u are kept in 8 bits, within 2^-4 of themselves, between the passes
    close = lambda a, b: float((a.double().cpu() - b).norm() / b.norm()) <= 2.0 ** -4
    assert close(xl.grad, dX)
    if not four:
        assert close(gul.grad, dGU) and close(dl.grad, dDN)


def test_serving_in_four_and_eight_bits(env):
    """A decode batch through 4-bit experts, rows as they are, in 8 and in 4 bits."""
    dev, tm = env
    N, H, O, E, k = 32, 128, 96, 8, 2
    x, w = rnd(1, N, H, dt=torch.bfloat16), rnd(2, E, O, H, scale=H ** -0.5)
    idx = torch.randint(0, E, (N, k), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    idx[5] = -1  # a padding token
    alpha = torch.rand(N, k, generator=torch.Generator().manual_seed(4))
    p = tm.mx4_pack(w.to(dev))
    wv = R.from_mx4(p.q.cpu(), p.scale.cpu())
    r = tm.moe_dispatch_fwd(x.to(dev), idx.to(dev), E)
    for rows, xv in ((r.xs, x.double()), (tm.act8_pack(r.xs), BR.act8(x)[2]),
                     (tm.mx4_pack(r.xs), R.from_mx4(*R.mx4(x)))):
        y = tm.moe_combine_fwd(tm.mx4_linear_fwd(rows, p, r.expert_offsets), r.entry_row, alpha.to(dev))
        torch.cuda.synchronize()
        ref = torch.zeros(N, O, dtype=torch.float64)
        tol = torch.zeros_like(ref)
        for t in range(N):
            for j in range(k):
                if idx[t, j] >= 0:
                    v, a = wv[idx[t, j]] @ xv[t], float(alpha[t, j])
                    ref[t] += a * v
                    tol[t] += a * (2.0 ** -8 * v.abs() + (WINDOW + 2 * H * R.U32) * (wv[idx[t, j]].abs() @ xv[t].abs()))
        BR.check("y", y, ref, tol + (2.0 ** -8 + 2.0 ** -14) * (ref.abs() + tol))
        assert not y[5].any()


def test_captured_and_replayed(env):
    """Forward and backward in one graph, over new rows, matrices and offsets."""
    dev, tm = env
    d, E, Rn, K, O = torch.bfloat16, 4, 1300, 96, 640
    bufs = [torch.zeros(s, dtype=t, device=dev) for s, t in
            (((Rn, K), d), ((E, O, K), d), ((Rn, O), d), ((E + 1,), torch.int32))]

    def step():
        x, w, dy, off = bufs
        y = tm.moe_linear_fwd(x, w, off)
        g = tm.moe_linear_bwd(dy, x, w, off)
        p = tm.mx4_pack(w)
        return [y, g.dx, g.dw, tm.mx4_linear_fwd(x, p, off), tm.mx4_linear_fwd(tm.mx4_pack(x), p, off),
                tm.mx4_linear_fwd(tm.act8_pack(x), p, off), tm.mx4_linear_bwd(dy, p, off)]

    def load(i):
        sizes = ([400, 0, 800, 100], [1300, 0, 0, 0], [325, 325, 325, 325], [0, 0, 0, 7])[i % 4]
        for b, v in zip(bufs, (rnd(i, Rn, K, dt=d), rnd(i + 50, E, O, K, dt=d), rnd(i + 90, Rn, O, dt=d),
                               offsets(sizes))):
            b.copy_(v)

    want = []
    for i in range(4):
        load(i)
        want.append([t.clone() for t in step()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in (1, 0, 2, 3, 1):
        load(i)
        for o in outs:
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want[i])), i
        torch.randn(1 << 16, device=dev).sum().item()


def test_functions_captured(env):
    dev, tm = env
    d, E, Rn, K, O = torch.bfloat16, 3, 100, 64, 72
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((Rn, K), (E, O, K), (Rn, O))))
    off = offsets([30, 0, 60]).to(dev)
    want = tm.moe_linear_bwd(dy, x, w, off)
    p = tm.mx4_pack(w)
    want4 = tm.mx4_linear_bwd(dy, p, off)
    a, b = leaves(x, w)
    c, = leaves(x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        tm.moe_linear(a, b, off).backward(dy)
        tm.mx4_linear(c, p, off).backward(dy)
    torch.cuda.synchronize()
    for t in (a, b, c):
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tm.moe_linear(a, b, off).backward(dy)
        tm.mx4_linear(c, p, off).backward(dy)
    for _ in range(3):
        for t in (a, b, c):
            t.grad.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        # a captured first gradient is stored, not added
        assert same(a.grad, want.dx) and same(b.grad, want.dw) and same(c.grad, want4)


def test_two_streams_at_once(env):
    """Calls on two streams, each with workspaces of its own, and a raw stream handle."""
    dev, tm = env
    d = torch.bfloat16
    S = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for i, (sizes, K, O) in enumerate((([900, 40, 100], 264, 520), ([700, 0, 341], 520, 264))):
        n = sum(sizes)
        x, w, dy = (rnd(10 * i + j, *s, dt=d).to(dev) for j, s in enumerate(((n, K), (3, O, K), (n, O))))
        off = offsets(sizes).to(dev)
        p = tm.mx4_pack(w) if K % 32 == 0 else None
        cases.append((x, w, dy, off, tm.moe_linear_fwd(x, w, off), tm.moe_linear_bwd(dy, x, w, off)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (x, w, dy, off, _, _) in enumerate(cases):
            st = S[i] if i else S[i].cuda_stream
            got[i].append((tm.moe_linear_fwd(x, w, off, stream=st), tm.moe_linear_bwd(dy, x, w, off, stream=st)))
    torch.cuda.synchronize()
    for i, (_, _, _, _, y, g) in enumerate(cases):
        for y2, g2 in got[i]:
            assert same(y, y2) and same(g.dx, g2.dx) and same(g.dw, g2.dw)


def test_buffers_of_the_caller(env):
    dev, tm = env
    d, sizes, K, O = torch.bfloat16, [50, 3], 64, 96
    off = offsets(sizes).to(dev)
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((60, K), (2, O, K), (60, O))))
    y, g = tm.moe_linear_fwd(x, w, off), tm.moe_linear_bwd(dy, x, w, off)
    wide = torch.full((60, O + 40), 5.0, dtype=d, device=dev)
    assert tm.moe_linear_fwd(x, w, off, y=wide[:, 16:16 + O]).data_ptr() == wide[:, 16:].data_ptr()
    dxw, dw = torch.full((60, K + 8), 5.0, dtype=d, device=dev), torch.empty_like(w)
    ws = torch.empty(tm.moe_linear_bwd_workspace_bytes(60, K, O, 2), dtype=torch.uint8, device=dev)
    tm.moe_linear_bwd(dy, x, w, off, dx=dxw[:, :K], dw=dw, workspace=ws)
    torch.cuda.synchronize()
    assert same(wide[:, 16:16 + O].contiguous(), y) and same(dxw[:, :K].contiguous(), g.dx) and same(dw, g.dw)
    assert bool((wide[:, :16] == 5).all()) and bool((wide[:, 16 + O:] == 5).all()) and bool((dxw[:, K:] == 5).all())
    p = tm.mx4_pack(w)
    ws = torch.empty(tm.mx4_linear_bwd_workspace_bytes(60, K, O, 2), dtype=torch.uint8, device=dev)
    dx = tm.mx4_linear_bwd(dy, p, off, workspace=ws, dx=dxw[:, :K])
    torch.cuda.synchronize()
    assert same(dx.contiguous(), tm.mx4_linear_bwd(dy, p, off))


def test_no_rows(env):
    dev, tm = env
    for d in DT.values():
        x, w, dy = torch.empty(0, 64, dtype=d, device=dev), rnd(1, 3, 32, 64, dt=d).to(dev), \
            torch.empty(0, 32, dtype=d, device=dev)
        off = torch.zeros(4, dtype=torch.int32, device=dev)
        assert tm.moe_linear_fwd(x, w, off).shape == (0, 32)
        g = tm.moe_linear_bwd(dy, x, w, off)
        torch.cuda.synchronize()
        assert g.dx.shape == (0, 64) and g.dw.shape == w.shape and not g.dw.any()
        p = tm.mx4_pack(w)
        assert tm.mx4_linear_fwd(x, p, off).shape == (0, 32)
        assert tm.mx4_linear_fwd(tm.mx4_pack(x), p, off).shape == (0, 32)
        assert tm.mx4_linear_bwd(dy, p, off).shape == (0, 64)
        assert tm.moe_linear_bwd(dy, x, w, off, need_dx=False, need_dw=False) == (None, None)


def test_gpu_refusals(env):
    dev, tm = env
    d = torch.bfloat16
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((10, 64), (2, 32, 64), (10, 32))))
    off = offsets([4, 5]).to(dev)
    p = tm.mx4_pack(w)
    xa, xm = tm.act8_pack(x), tm.mx4_pack(x)
    ws = torch.empty(64, dtype=torch.uint8, device=dev)
    bad = [
        (ValueError, lambda: tm.moe_linear_fwd(x, w)),                      # two experts, no offsets
        (ValueError, lambda: tm.moe_linear_fwd(x, w, off[:2])),
        (TypeError, lambda: tm.moe_linear_fwd(x, w, off.long())),
        (ValueError, lambda: tm.moe_linear_fwd(x, w, off.cpu())),
        (ValueError, lambda: tm.moe_linear_fwd(x[:, :32], w, off)),
        (TypeError, lambda: tm.moe_linear_fwd(x, w.float(), off)),
        (TypeError, lambda: tm.moe_linear_fwd(x.half(), w.half(), off)),
        (ValueError, lambda: tm.moe_linear_fwd(x[None], w, off)),
        (ValueError, lambda: tm.moe_linear_fwd(x.t().contiguous().t(), w, off)),
        (ValueError, lambda: tm.moe_linear_fwd(x, w.transpose(1, 2).contiguous().transpose(1, 2), off)),
        (tm.TopmoeError, lambda: tm.moe_linear_fwd(x[:, :60].contiguous(), w[..., :60].contiguous(), off)),
        (tm.TopmoeError, lambda: tm.moe_linear_fwd(torch.empty(10, 68, dtype=d, device=dev)[:, :64], w, off)),
        (tm.TopmoeError, lambda: tm.moe_linear_fwd(torch.empty(700, dtype=d, device=dev)[4:644].view(10, 64), w, off)),
        (ValueError, lambda: tm.moe_linear_fwd(x, w, off, y=torch.empty(10, 40, dtype=d, device=dev))),
        (TypeError, lambda: tm.moe_linear_fwd(x, w, off, y=torch.empty(10, 32, device=dev))),
        (ValueError, lambda: tm.moe_linear_bwd(dy[:9], x, w, off)),
        (TypeError, lambda: tm.moe_linear_bwd(dy, None, w, off)),
        (TypeError, lambda: tm.moe_linear_bwd(dy, x, None, off)),
        (ValueError, lambda: tm.moe_linear_bwd(dy, x, w[:, :16].contiguous(), off)),
        (ValueError, lambda: tm.moe_linear_bwd(dy, x, w, off, workspace=ws)),
        (ValueError, lambda: tm.mx4_linear_bwd(dy, p, off, workspace=ws)),
        (ValueError, lambda: tm.mx4_linear_bwd(dy[:, :24].contiguous(), p, off)),
        (tm.TopmoeError, lambda: tm.mx4_pack(x[:, :60].contiguous())),
        (TypeError, lambda: tm.mx4_pack(x.half())),
        (ValueError, lambda: tm.mx4_pack(torch.zeros(64, device=dev))),
        (ValueError, lambda: tm.mx4_pack(w.transpose(0, 1))),
        (ValueError, lambda: tm.mx4_unpack(tm.Mx4(p.q, p.scale[:1]))),
        (TypeError, lambda: tm.mx4_unpack(tm.Mx4(p.q.to(torch.int8), p.scale))),
        (ValueError, lambda: tm.mx4_unpack(p, x=torch.empty(2, 32, 60, dtype=d, device=dev))),
        (TypeError, lambda: tm.mx4_unpack(p, dtype=torch.float16)),
        (TypeError, lambda: tm.mx4_linear_fwd(x, w, off)),                  # not in 4 bits
        (TypeError, lambda: tm.mx4_linear_fwd(x, p, off, dtype=torch.float32)),
        (ValueError, lambda: tm.mx4_linear_fwd(x[:, :32], p, off)),
        (ValueError, lambda: tm.mx4_linear_fwd(tm.Act8(xa.q, xa.scale[:5]), p, off)),
        (TypeError, lambda: tm.mx4_linear_fwd(tm.Act8(xa.q.view(torch.uint8), xa.scale), p, off)),
        (ValueError, lambda: tm.mx4_linear_fwd(xm, tm.mx4_pack(w[..., :32].contiguous()), off)),
        (tm.TopmoeError, lambda: tm.mx4_linear_fwd(x[:, :40].contiguous(), tm.mx4_pack(w[..., :40].contiguous()), off)),
        (TypeError, lambda: tm.mx4_linear_fwd(xm, p, off, dtype=torch.float16)),
    ]
    for i, (err, f) in enumerate(bad):
        with pytest.raises(err):
            f()
            pytest.fail(f"call {i} was not refused")


def test_stage_events(env):
    dev, tm = env
    d = torch.bfloat16
    x, w, dy = (rnd(i, *s, dt=d).to(dev) for i, s in enumerate(((1300, 64), (4, 6464, 64), (1300, 6464))))
    off = offsets([1000, 100, 100, 100]).to(dev)
    ev = tm.StageEvents(2)
    tm.moe_linear_bwd(dy, x, w, off, stage_events=ev)
    t = ev.elapsed_ms()
    assert len(t) == 2 and all(0 < v < 100 for v in t)
    tm.moe_linear_bwd(dy, x, w, off, need_dx=False, stage_events=ev)
    t = ev.elapsed_ms()
    assert t[1] > 0
    p = tm.mx4_pack(w)
    tm.mx4_linear_bwd(dy, p, off, stage_events=ev)
    assert all(0 < v < 100 for v in ev.elapsed_ms())
    with pytest.raises(ValueError, match="stages"):
        tm.mx4_linear_bwd(dy, p, off, stage_events=tm.StageEvents(1))
    one = tm.StageEvents(1)
    tm.mx4_linear_fwd(x, p, off, stage_events=one)
    assert one.elapsed_ms()[0] > 0


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes,K,O", [
    ([700] + [100] * 7, 264, 392), ([0] * 7 + [1400], 264, 392), ([650] + [43] * 15, 264, 392),
    ([1] * 15 + [1300], 136, 264), ([600] + [26] * 23, 264, 392), ([500] + [10] * 63, 136, 264),
    ([3200] + [457] * 7, 264, 392), ([5000] + [1000] * 15, 136, 264)])
def test_dw_of_skewed_experts(env, sizes, K, O, dt):
    """One expert with most of the rows beside 7, 15 and more others, whole sums and parts."""
    dev, tm = env
    d, n = DT[dt], sum(sizes)
    announce(f"dw of {len(sizes)} experts, {max(sizes)} of {n} rows in one, {K} x {O} {dt}")
    x, dy, w = rnd(1, n, K, dt=d), rnd(2, n, O, dt=d), torch.empty(len(sizes), O, K, dtype=d, device=dev)
    off = offsets(sizes).to(dev)
    dw = tm.moe_linear_bwd(dy.to(dev), x.to(dev), w, off, need_dx=False).dw
    torch.cuda.synchronize()
    ref = R.grouped_dw(dy, x, sizes)
    BR.check("dw", dw, ref, R.tol(ref, R.grouped_dw(dy.abs(), x.abs(), sizes), max(sizes), d))
    assert same(dw, tm.moe_linear_bwd(dy.to(dev), x.to(dev), w, off, need_dx=False).dw)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_bwd_takes_its_dtypes_workspace(env, dt):
    """As many bytes as the dtype needs are enough, and the front end takes no more."""
    dev, tm = env
    d = DT[dt]
    for sizes, K, O in (([512] * 8, 264, 392), ([2400, 0, 260, 300, 280, 310, 250, 1000], 136, 72), ([20], 64, 6464)):
        n, E = sum(sizes), len(sizes)
        x, dy = rnd(1, n, K, dt=d).to(dev), rnd(2, n, O, dt=d).to(dev)
        w, off = rnd(3, E, O, K, dt=d).to(dev), offsets(sizes).to(dev)
        need = tm.moe_linear_bwd_workspace_bytes(n, K, O, E, d)
        ws = torch.full((need + 4096,), 7, dtype=torch.uint8, device=dev)
        g = tm.moe_linear_bwd(dy, x, w, off, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((ws[need:] == 7).all())
        del ws
        # bytes asked for (allocated ones count the allocator's blocks, up to 1 MiB larger)
        before = torch.cuda.memory_stats()["requested_bytes.all.current"]
        torch.cuda.reset_peak_memory_stats()
        h = tm.moe_linear_bwd(dy, x, w, off)
        torch.cuda.synchronize()
        asked = torch.cuda.memory_stats()["requested_bytes.all.peak"] - before
        assert asked == (x.numel() + w.numel()) * x.element_size() + need
        assert same(g.dx, h.dx) and same(g.dw, h.dw)


def test_four_bits_on_two_streams_at_once(env):
    """4-bit products and gradients on two streams (whose gradients keep unpacked matrices and parts in
    workspaces from launch to launch), one of them a raw handle: the bits of one after the other."""
    dev, tm = env
    S = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for i, (sizes, K, O) in enumerate((([900, 40, 100], 288, 544), ([300, 0, 141], 544, 288))):
        n, off = sum(sizes), offsets(sizes).to(dev)
        p = tm.mx4_pack(rnd(10 * i, 3, O, K).to(dev))
        for d in DT.values():
            cases.append((i, rnd(10 * i + 1, n, K, dt=d).to(dev), rnd(10 * i + 2, n, O, dt=d).to(dev), p, off))

    def step(x, dy, p, off, **on):
        a8, m4 = tm.act8_pack(x, **on), tm.mx4_pack(x, **on)
        return [tm.mx4_linear_fwd(x, p, off, **on), tm.mx4_linear_fwd(a8, p, off, dtype=x.dtype, **on),
                tm.mx4_linear_fwd(m4, p, off, dtype=x.dtype, **on), tm.mx4_linear_bwd(dy, p, off, **on),
                tm.mx4_unpack(p, dtype=x.dtype, **on)]

    want = [step(*c[1:]) for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i, *c in cases:
            got.append(step(*c, stream=S[i] if i else S[i].cuda_stream))
    torch.cuda.synchronize()
    for j, outs in enumerate(got):
        assert all(same(a, b) for a, b in zip(outs, want[j % len(cases)])), j
