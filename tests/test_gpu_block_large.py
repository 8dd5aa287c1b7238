"""The block operators past 2^31 elements and past one launch's share of rows:
mostly zero tensors with a few rows of values, of which the ends, the rows next
to 2^31 elements and the rows next to a launch's last are looked at."""
import pytest
import torch

import block_ref as R
from gpu_util import announce, torch_dev

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
F32 = torch.float32


@pytest.fixture(scope="module")
def env():
    torch_, dev = torch_dev()
    import top_moe_layer_amd as tm

    tm.lib()
    if torch.cuda.get_device_properties(0).total_memory < 128 << 30:
        pytest.skip("needs 128 GiB of GPU memory")
    yield dev, tm
    torch.cuda.empty_cache()


def rows_to_check(N, H, *extra):
    """First, last, and those around 2^31 elements and each of `extra`."""
    at = {0, 1, N - 2, N - 1}
    for m in ((1 << 31) // H, (1 << 32) // H) + extra:
        at |= {m - 1, m, m + 1}
    return torch.tensor(sorted(r for r in at if 0 <= r < N))


def sparse(dev, N, H, at, seed, dt=BF):
    """[N, H] of zeros but for the rows `at`; those rows on the CPU."""
    v = torch.randn(len(at), H, generator=torch.Generator().manual_seed(seed)).to(dt)
    x = torch.zeros(N, H, dtype=dt, device=dev)
    x[at.to(dev)] = v.to(dev)
    return x, v


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


@pytest.mark.parametrize("N,C,dt", [(70000, 32768, BF), (1 << 20, 8200, BF), (20000, 4104, F32)])
def test_act8_large(env, N, C, dt):
    """The second has more than 2^30 pieces of 8: two launches."""
    dev, tm = env
    announce(f"act8 {N} x {C} {dt}")
    pieces = -(-C // 32) * 4
    at = rows_to_check(N, C, (1 << 30) // pieces)
    x, v = sparse(dev, N, C, at, 1, dt)
    a = tm.act8_pack(x)
    y = tm.act8_unpack(a.q, a.scale, dtype=dt)
    torch.cuda.synchronize()
    codes, scale, _ = R.act8(v)
    d = at.to(dev)
    assert torch.equal(a.q.view(torch.uint8)[d].cpu().long(), codes)
    assert torch.equal(a.scale[d].cpu(), scale)
    other = tm.act8_unpack(a.q[d].contiguous(), a.scale[d].contiguous(), dtype=dt)
    assert torch.equal(bits(y[d]), bits(other))
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(y[d]))


@pytest.mark.parametrize("N,C,dt", [(70000, 32768, BF), (20000, 4104, F32)])
def test_swiglu_act8_large(env, N, C, dt):
    dev, tm = env
    announce(f"swiglu_act8 {N} x {C} {dt}")
    at = rows_to_check(N, C)
    g, gv = sparse(dev, N, C, at, 1, dt)
    u, uv = sparse(dev, N, C, at, 2, dt)
    d = at.to(dev)
    o = tm.swiglu_act8_fwd(g, u)
    s = tm.swiglu_act8_fwd(gv.to(dev), uv.to(dev))
    assert torch.equal(bits(o.h[d]), bits(s.h)) and torch.equal(bits(o.g8.q[d]), bits(s.g8.q))
    b = tm.swiglu_act8_bwd(u, o.g8, o.u8)
    t = tm.swiglu_act8_bwd(uv.to(dev), s.g8, s.u8)
    torch.cuda.synchronize()
    for big, small in ((b.dg, t.dg), (b.du, t.du), (b.h, t.h)):
        assert torch.equal(bits(big[d]), bits(small))


@pytest.mark.parametrize("N,H,dt", [(140000, 16384, BF), ((1 << 22) + 100, 8, BF),
                                    (20000, 4104, F32), (40000, 1000, F32), (300000, 64, F32)])
def test_norms_large(env, N, H, dt):
    """The second has more than 2^22 rows: three launches of the forward."""
    dev, tm = env
    announce(f"norms {N} x {H} {dt}")
    at = rows_to_check(N, H, 1 << 21)
    d = at.to(dev)
    y, yv = sparse(dev, N, H, at, 1, dt)
    r, rv = sparse(dev, N, H, at, 2, dt)
    w = torch.rand(H, generator=torch.Generator().manual_seed(3)).to(dt).to(dev)
    kw = dict(gate=w, next_w=w, residual_scale=0.5)
    o = tm.block_postnorm_fwd(y, r, w, **kw)
    s = tm.block_postnorm_fwd(yv.to(dev), rv.to(dev), w, **kw)
    torch.cuda.synchronize()
    assert torch.equal(bits(o.out[d]), bits(s.out)) and torch.equal(bits(o.n[d]), bits(s.n))
    assert torch.equal(o.rstd[d], s.rstd) and torch.equal(o.next_rstd[d], s.next_rstd)
    b = tm.block_postnorm_bwd(r, y, w, rstd=o.rstd, dn=y, out=o.out, next_rstd=o.next_rstd, **kw)
    t = tm.block_postnorm_bwd(rv.to(dev), yv.to(dev), w, rstd=s.rstd, dn=yv.to(dev), out=s.out,
                              next_rstd=s.next_rstd, **kw)
    torch.cuda.synchronize()
    assert torch.equal(bits(b.dy[d]), bits(t.dy)) and torch.equal(bits(b.dresidual[d]), bits(t.dresidual))
    for n in ("dw", "dgate", "dnext_w"):  # the other rows add zeros, in another order of sums
        big, small = getattr(b, n).double().cpu(), getattr(t, n).double().cpu()
        assert bool(((big - small).abs() <= 2.0 ** -7 * small.abs() + 1e-5 * small.abs().max()).all()), n


@pytest.mark.parametrize("N,H,dt", [(70000, 16384, BF), (20000, 4104, F32)])
def test_rows_large(env, N, H, dt):
    """Rows past 2^31 elements both ways, k = 2, every entry kept."""
    dev, tm = env
    E, k = 7, 2
    announce(f"rows {N} x {H}, k = {k} {dt}")
    at = rows_to_check(N, H, 65536)
    x, v = sparse(dev, N, H, at, 1, dt)
    idx = torch.randint(0, E, (N, k), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    o = tm.moe_dispatch_fwd(x, idx.to(dev), E)
    torch.cuda.synchronize()
    er = o.entry_row[at.to(dev)].long()
    for j in range(k):
        assert torch.equal(bits(o.xs[er[:, j]]), bits(v))
    alpha = torch.rand(N, k, device=dev)
    y = tm.moe_combine_fwd(o.xs, o.entry_row, alpha)
    c = tm.moe_combine_bwd(x, o.xs, o.entry_row, alpha)
    dx = tm.moe_dispatch_bwd(o.xs, o.entry_row)
    torch.cuda.synchronize()
    a, f = alpha[at.to(dev)].cpu().double(), v.double()
    half = R.half_step(dt)
    ref = a.sum(-1, keepdim=True) * f
    R.check("y", y[at.to(dev)], ref, (half + 4 * R.U32) * ref.abs())
    R.check("dx", dx[at.to(dev)], 2 * f, half * 2 * f.abs())
    for j in range(k):
        R.check("dys", c.dys[er[:, j]], a[:, j, None] * f, (half + R.U32) * (a[:, j, None] * f).abs())
    sq = f.square().sum(-1, keepdim=True)
    R.check("dalpha", c.dalpha[at.to(dev)], sq.expand(-1, k), ((H / 64 + 16) * R.U32 * sq).expand(-1, k))


def test_entries_past_one_launch(env):
    """More than 2^24 entries (two launches of the combine's gradient), one chunk count past 256 x 1024."""
    dev, tm = env
    N, H, E = (1 << 24) + 77, 8, 200
    announce(f"{N} entries")
    g = torch.Generator(device=dev).manual_seed(1)
    idx = torch.randint(-1, E, (N, 1), generator=g, device=dev, dtype=torch.int32)
    x = torch.randn(N, H, generator=g, device=dev, dtype=torch.float32).to(BF)
    o = tm.moe_dispatch_fwd(x, idx, E)
    torch.cuda.synchronize()
    key = torch.where(idx[:, 0] < 0, E, idx[:, 0])
    order = torch.argsort(key, stable=True)
    kept = int((idx >= 0).sum())
    assert int(o.expert_offsets[E]) == kept
    assert torch.equal(o.row_entry[:kept].long(), order[:kept])
    assert bool((o.row_entry[kept:] == -1).all())
    assert torch.equal(o.xs[:kept], x[order[:kept]]) and not o.xs[kept:].any()
    assert bool(((o.entry_row[:, 0] >= 0) == (idx[:, 0] >= 0)).all())
    alpha = torch.rand(N, 1, generator=g, device=dev)
    c = tm.moe_combine_bwd(x, o.xs, o.entry_row, alpha)
    torch.cuda.synchronize()
    want = torch.where(idx >= 0, x.float().square().sum(-1, keepdim=True), 0.0)
    assert bool(((c.dalpha - want).abs() <= 16 * R.U32 * want).all())
    assert not c.dys[kept:].any()
    ref = (alpha * x.float()).to(BF)
    assert torch.equal(c.dys[:kept], ref[order[:kept]])


def test_gradients_may_be_written_over_their_inputs(env):
    """dresidual over dout, dx over the residual stream's gradient (C ABI)."""
    dev, tm = env
    from top_moe_layer_amd import _binding as B

    N, H = 300, 200
    r = lambda seed, *s: torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(BF).to(dev)
    x, w, dn, dres = r(1, N, H), r(2, H), r(3, N, H), r(4, N, H)
    f = tm.block_prenorm_fwd(x, w)
    want = tm.block_prenorm_bwd(dn, x, w, f.rstd, dresidual=dres)
    ws = torch.empty(tm.block_norm_bwd_workspace_bytes(N, H), dtype=torch.uint8, device=dev)
    over, dw = dres.clone(), torch.empty_like(w)
    s = torch.cuda.current_stream().cuda_stream
    B.check(B.lib().block_prenorm_bwd(dn.data_ptr(), x.data_ptr(), w.data_ptr(), f.rstd.data_ptr(),
                                      over.data_ptr(), N, H, B.DTYPE_BF16, over.data_ptr(),
                                      dw.data_ptr(), ws.data_ptr(), ws.numel(), s, None))
    torch.cuda.synchronize()
    assert torch.equal(bits(over), bits(want.dx)) and torch.equal(bits(dw), bits(want.dw))
    p = tm.block_postnorm_fwd(x, dn, w, next_w=w)
    want = tm.block_postnorm_bwd(dres, x, w, rstd=p.rstd, dn=dn, out=p.out, next_w=w,
                                 next_rstd=p.next_rstd)
    over, dy, dw2 = dres.clone(), torch.empty_like(x), torch.empty_like(w)
    B.check(B.lib().block_postnorm_bwd(
        over.data_ptr(), dn.data_ptr(), x.data_ptr(), p.out.data_ptr(), w.data_ptr(), None,
        w.data_ptr(), p.rstd.data_ptr(), p.next_rstd.data_ptr(), N, H, 0, 1, 1.0, B.DTYPE_BF16,
        dy.data_ptr(), over.data_ptr(), dw.data_ptr(), None, dw2.data_ptr(), ws.data_ptr(),
        ws.numel(), s, None))
    torch.cuda.synchronize()
    assert torch.equal(bits(over), bits(want.dresidual)) and torch.equal(bits(dy), bits(want.dy))
    assert torch.equal(bits(dw), bits(want.dw)) and torch.equal(bits(dw2), bits(want.dnext_w))
