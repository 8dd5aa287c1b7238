"""Products by expert and 4-bit matrices past 2^31 elements and bytes, on sampled rows."""
import pytest
import torch

import block_ref as BR
import linear_ref as R
from gpu_util import announce, torch_dev

pytestmark = pytest.mark.gpu
U32 = BR.U32


@pytest.fixture(scope="module")
def env():
    torch_, dev = torch_dev()
    import top_moe_layer_amd as tm

    tm.lib()
    return dev, tm


def fill(shape, dev, seed, scale=1.0, dt=torch.bfloat16):
    g = torch.Generator(device=dev).manual_seed(seed)
    t = torch.empty(shape, dtype=dt, device=dev)
    flat = t.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=g, device=dev).mul_(scale)
    return t


def close(got, a, b, terms, extra=0.0):
    """got = a b^T, from operands in 64 bits."""
    a, b = a.double().cpu(), b.double().cpu()
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    BR.check("sample", got, ref, R.tol(ref, mag, terms, got.dtype) + extra * mag)


def test_many_rows(env):
    """2^31 elements of x, of y and of their gradients."""
    dev, tm = env
    Rn, K, O = (1 << 20) + 300, 2048, 2056
    announce(f"linear {Rn} rows, {K} -> {O}")
    x, w = fill((Rn, K), dev, 1), fill((2, O, K), dev, 2, K ** -0.5)
    off = torch.tensor([0, Rn // 2 + 77, Rn - 100], dtype=torch.int32, device=dev)
    rows = torch.tensor([0, 1, Rn // 2 + 76, Rn // 2 + 77, Rn - 200, Rn - 101])
    expert = [0, 0, 0, 1, 1, 1]
    y = tm.moe_linear_fwd(x, w, off)
    torch.cuda.synchronize()
    for r, e in zip(rows.tolist(), expert):
        close(y[r:r + 1], x[r:r + 1], w[e], K)
    assert not y[Rn - 100:].any()
    g = tm.moe_linear_bwd(y, x, w, off)  # y as the gradient
    torch.cuda.synchronize()
    for r, e in zip(rows.tolist(), expert):
        close(g.dx[r:r + 1], y[r:r + 1], w[e].T, O)
    assert not g.dx[Rn - 100:].any()
    first = Rn // 2 + 77
    want = torch.zeros(16, 32, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(want)
    for a in range(0, first, 1 << 16):
        b = min(first, a + (1 << 16))
        p, q = y[a:b, 2040:2056].double(), x[a:b, :32].double()
        want += p.T @ q
        mag += p.abs().T @ q.abs()
    want, mag = want.cpu(), mag.cpu()
    BR.check("dw", g.dw[0, 2040:2056, :32], want, R.tol(want, mag, first, torch.bfloat16))
    del g, y
    p = tm.mx4_pack(w)
    wv = tm.mx4_unpack(p, dtype=torch.float32)
    for rows_, xv in ((x, x), (tm.mx4_pack(x), None)):
        y = tm.mx4_linear_fwd(rows_, p, off)
        torch.cuda.synchronize()
        for r, e in zip(rows.tolist(), expert):
            row = x[r:r + 1] if xv is not None else R.from_mx4(*R.mx4(x[r:r + 1].cpu()))
            close(y[r:r + 1], row, wv[e], K)
        del y


def test_many_weights(env):
    """More than 2^31 elements of the experts' matrices, and of their gradient; decode-sized and more rows."""
    dev, tm = env
    E, O, K = 256, 4104, 2080
    announce(f"linear {E} experts, {K} -> {O}")
    w = fill((E, O, K), dev, 1, K ** -0.5)
    for n in (1, 40):
        Rn = E * n
        x = fill((Rn, K), dev, 2)
        off = (torch.arange(E + 1, device=dev) * n).to(torch.int32)
        y = tm.moe_linear_fwd(x, w, off)
        torch.cuda.synchronize()
        for e in (0, 1, 251, 255):
            close(y[e * n:e * n + 1, -40:], x[e * n:e * n + 1], w[e, -40:], K)
        dx = tm.moe_linear_bwd(y, None, w, off, need_dw=False).dx
        torch.cuda.synchronize()
        for e in (0, 255):
            close(dx[e * n:e * n + 1, -40:], y[e * n:e * n + 1], w[e, :, -40:].T, O)
        dw = tm.moe_linear_bwd(y, x, w, off, need_dx=False).dw
        torch.cuda.synchronize()
        for e in (0, 255):
            close(dw[e, -24:], y[e * n:e * n + n, -24:].T, x[e * n:e * n + n].T, n)
        del dw, dx
    p = tm.mx4_pack(w)
    del w
    for n in (1, 40):
        x = fill((E * n, K), dev, 3)
        off = (torch.arange(E + 1, device=dev) * n).to(torch.int32)
        for arg in (x, tm.mx4_pack(x)):
            y = tm.mx4_linear_fwd(arg, p, off)
            torch.cuda.synchronize()
            for e in (0, 255):
                row = x[e * n:e * n + 1].cpu()
                row = row if arg is x else R.from_mx4(*R.mx4(row))
                close(y[e * n:e * n + 1], row, R.from_mx4(p.q[e].cpu(), p.scale[e].cpu()), K)
        dx = tm.mx4_linear_bwd(y, p, off)
        torch.cuda.synchronize()
        close(dx[-1:], y[-1:], R.from_mx4(p.q[255].cpu(), p.scale[255].cpu()).T, O)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_pack_large(env, dt):
    dev, tm = env
    Rn, C = (1 << 21) + 5, 1032
    announce(f"mx4 {Rn} x {C} {dt}")
    x = fill((Rn, C), dev, 1, dt=dt)
    p = tm.mx4_pack(x)
    y = tm.mx4_unpack(p, dtype=dt)
    torch.cuda.synchronize()
    for r in (0, 1, Rn // 2, Rn - 2, Rn - 1):
        q, s = R.mx4(x[r:r + 1].cpu())
        assert torch.equal(p.q[r:r + 1].cpu(), q) and torch.equal(p.scale[r:r + 1].cpu(), s)
        assert torch.equal(y[r:r + 1].cpu().double(), R.from_mx4(q, s))
