"""The block operators on the GPU against their 64-bit definitions (block_ref):
rows by expert and back, norms with gate and residual, activations in 8 bits.

Tolerances count roundings.  An output of the dtype is off by half a step of
it; before that, sums of L terms in 32 bits are off by at most L * 2^-24 of the
sum of the terms' magnitudes, with L the longest chain of additions."""
import math

import pytest
import torch

import block_ref as R
from gpu_util import announce, torch_dev

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def env():
    torch_, dev = torch_dev()
    import top_moe_layer_amd as tm

    tm.lib()
    return dev, tm


def rnd(seed, *shape, dt=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dt)


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


# ------------------------------------------------------------ rows by expert
ROUTES = [  # N, H, E, k, capacity factor, share of padding tokens, one expert takes everything
    (1, 8, 1, 1, 0.0, 0.0, False),
    (1, 2048, 16, 2, 0.0, 0.0, False),
    (5, 24, 3, 3, 0.0, 0.4, False),
    (32, 768, 256, 8, 0.0, 0.0, False),
    (33, 40, 256, 256, 0.5, 0.1, False),
    (128, 64, 8, 8, 1.0, 0.0, True),
    (257, 4096, 8, 4, 1.0, 0.1, False),  # blocks of two tokens, the last of one
    (16384, 8, 7, 2, 1.0, 0.1, False),   # the last one-launch size
    (128, 16, 256, 256, 0.0, 0.0, False),
    (16385, 8, 7, 2, 1.0, 0.1, False),   # the first with three launches
    (90, 131072, 4, 3, 1.0, 0.1, False),  # few entries of long rows: bf16 one launch, fp32 three
    (700, 104, 5, 2, 0.0, 0.0, False),
    (700, 104, 5, 2, 0.01, 0.3, True),
    (701, 200, 5, 2, 0.0, 0.1, False),  # parts of a wavefront a row, or a whole one
    (61, 128, 6, 3, 1.0, 0.1, False),
    (61, 256, 6, 3, 1.0, 0.1, False),
    (61, 264, 6, 3, 1.0, 0.1, False),
    (3001, 16, 64, 6, 1.25, 0.05, False),
    (2500, 8, 256, 4, 1.0, 0.0, True),
    (40000, 8, 2, 1, 0.0, 0.0, False),
    (300000, 8, 255, 1, 0.75, 0.1, False),  # chunks of more than 1024 entries
]


def route(seed, N, E, k, pad, one):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, E, (N, k), generator=g, dtype=torch.int32)  # an expert may come twice
    if one:
        idx[torch.rand(N, k, generator=g) < 0.9] = E - 1
    idx[torch.rand(N, generator=g) < pad] = -1
    if pad:
        idx[0, 0] = E  # just outside
        if N > 1:
            idx[1, k - 1] = -2 ** 31
    return idx


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,E,k,cf,pad,one", ROUTES)
def test_dispatch(env, N, H, E, k, cf, pad, one, dt):
    dev, tm = env
    announce(f"dispatch N={N} H={H} E={E} k={k} cf={cf} {dt}")
    idx = route(N + E, N, E, k, pad, one)
    x = rnd(1, N, H, dt=DT[dt])
    o = tm.moe_dispatch_fwd(x.to(dev), idx.to(dev), E, capacity_factor=cf)
    torch.cuda.synchronize()
    offsets, row_entry, entry_row = R.rows_of(idx.tolist(), E, cf)
    assert o.expert_offsets.tolist() == offsets
    assert o.entry_row.flatten().tolist() == entry_row
    assert o.row_entry.tolist() == row_entry
    want = torch.zeros(N * k, H, dtype=DT[dt])
    kept = offsets[-1]
    want[:kept] = x[torch.tensor(row_entry[:kept], dtype=torch.long) // k]
    assert torch.equal(bits(o.xs.cpu()), bits(want))


@pytest.mark.parametrize("N,E,k,cf", [(50, 10, 2, 1.2), (50, 10, 2, 0.6), (500, 8, 2, 1.2),
                                      (500, 8, 2, 1.6), (17000, 10, 2, 1.1)])
def test_dispatch_capacity_factors_between_floats(env, N, E, k, cf):
    """Factors whose product is a whole number, and which a float exceeds: the C entry point takes
    the float's own value, the front end the factor it is given."""
    dev, tm = env
    from top_moe_layer_amd import _binding as B

    announce(f"dispatch capacity N={N} E={E} k={k} factor {cf}")
    g = torch.Generator().manual_seed(N)
    idx = torch.where(torch.rand(N, k, generator=g) < 0.7, 1, 3).to(torch.int32)
    x, on = rnd(1, N, 8).to(dev), idx.to(dev)
    o = tm.moe_dispatch_fwd(x, on, E, capacity_factor=cf)
    torch.cuda.synchronize()
    want = R.rows_of(idx.tolist(), E, cf)
    assert (o.expert_offsets.tolist(), o.row_entry.tolist(), o.entry_row.flatten().tolist()) == want
    ws = torch.empty(tm.moe_dispatch_workspace_bytes(N, E, k), dtype=torch.uint8, device=dev)
    single = float(torch.tensor(cf, dtype=torch.float32))
    st = B.lib().moe_dispatch_fwd(x.data_ptr(), on.data_ptr(), N, 8, E, k, cf, B.DTYPE_FP32,
                                  o.xs.data_ptr(), o.expert_offsets.data_ptr(),
                                  o.row_entry.data_ptr(), o.entry_row.data_ptr(), ws.data_ptr(),
                                  ws.numel(), torch.cuda.current_stream().cuda_stream, None)
    torch.cuda.synchronize()
    assert st == B.OK
    assert o.expert_offsets.tolist() == R.rows_of(idx.tolist(), E, single)[0] != want[0]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,E,k,cf,pad,one", [r for r in ROUTES if r[0] * r[1] * r[3] < 1 << 21])
def test_back_to_tokens(env, N, H, E, k, cf, pad, one, dt):
    """dispatch's gradient, combine and combine's gradient; rows and weights of
    entries that are not kept hold NaN or infinity."""
    dev, tm = env
    announce(f"combine N={N} H={H} E={E} k={k} cf={cf} {dt}")
    d, half = DT[dt], R.half_step(DT[dt])
    idx = route(N + E, N, E, k, pad, one)
    offsets, row_entry, er = R.rows_of(idx.tolist(), E, cf)
    kept = offsets[-1]
    er = torch.tensor(er, dtype=torch.int32).reshape(N, k)
    rows = rnd(2, N * k, H, dt=d)
    rows[kept:] = math.nan
    alpha = torch.rand(N, k, generator=torch.Generator().manual_seed(3))
    alpha[er < 0] = math.inf
    res, dy = rnd(4, N, H, dt=d), rnd(5, N, H, dt=d)
    use = (er >= 0)
    at = torch.where(use, er, torch.zeros_like(er)).long()
    terms = torch.where(use[..., None], rows[at].double(), torch.zeros(1, dtype=torch.float64))
    al = torch.where(use, alpha, torch.zeros_like(alpha)).double()

    got = tm.moe_dispatch_bwd(rows.to(dev), er.to(dev))
    ref = terms.sum(1)
    R.check("dx", got, ref, half * ref.abs() + (k + 1) * R.U32 * terms.abs().sum(1))

    for r in (None, res):
        got = tm.moe_combine_fwd(rows.to(dev), er.to(dev), alpha.to(dev),
                                 residual=None if r is None else r.to(dev))
        t = al[..., None] * terms
        base = 0.0 if r is None else r.double()
        ref, mag = t.sum(1) + base, t.abs().sum(1) + (0.0 if r is None else base.abs())
        R.check("y", got, ref, half * ref.abs() + (k + 2) * R.U32 * mag)
    y = res.to(dev).clone()  # the residual's own memory
    tm.moe_combine_fwd(rows.to(dev), er.to(dev), alpha.to(dev), residual=y, y=y)
    assert torch.equal(bits(y), bits(got))

    o = tm.moe_combine_bwd(dy.to(dev), rows.to(dev), er.to(dev), alpha.to(dev))
    torch.cuda.synchronize()
    want = torch.zeros(N * k, H, dtype=torch.float64)
    want[er[use].long()] = (al[..., None] * dy.double()[:, None])[use]
    R.check("dys", o.dys, want, (half + R.U32) * want.abs())
    prod = terms * dy.double()[:, None]
    R.check("dalpha", o.dalpha, prod.sum(-1),
            (H / 64 + 16) * R.U32 * prod.abs().sum(-1))


def test_entry_rows_out_of_range(env):
    """Row ids that no dispatch writes add nothing and touch nothing."""
    dev, tm = env
    N, k, H = 4, 2, 16
    er = torch.tensor([[0, 9], [1, 2 ** 31 - 1], [-2 ** 31, 2], [3, -8]], dtype=torch.int32)
    rows, dy = rnd(1, N * k, H), rnd(2, N, H)
    alpha = torch.ones(N, k)
    got = tm.moe_combine_fwd(rows.to(dev), er.to(dev), alpha.to(dev))
    assert torch.equal(got.cpu(), rows[:4])
    o = tm.moe_combine_bwd(dy.to(dev), rows.to(dev), er.to(dev), alpha.to(dev))
    torch.cuda.synchronize()
    assert torch.equal(o.dys[:4].cpu(), dy)
    assert float(o.dys[7].abs().max()) == 0.0
    assert (o.dalpha.cpu()[er < 0] == 0).all() and (o.dalpha.cpu()[er >= 8] == 0).all()


# ------------------------------------------------------------ norms
def depth(H):
    """Longest chain of additions in a row's sum: a thread's channels, then lanes and wavefronts."""
    return H / 64 + 8 + 6 + 16


NORMS = [(1, 8), (3, 24), (7, 200), (5, 512), (2, 520), (100, 768), (9, 1000), (4, 2048),
         (3, 2056), (2, 4096), (3, 6008), (2, 8192), (2, 8200), (2, 16384)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H", NORMS + [(1100, 64), (2051, 40)])
def test_prenorm(env, N, H, dt):
    dev, tm = env
    announce(f"prenorm N={N} H={H} {dt}")
    d, half, eps = DT[dt], R.half_step(DT[dt]), 1e-5
    x, w = rnd(1, N, H, dt=d, scale=2.0), rnd(2, H, dt=d) + 1
    x[0] = 0  # rstd = 1 / sqrt(eps)
    dn, dres = rnd(3, N, H, dt=d), rnd(4, N, H, dt=d)
    K = depth(H)
    o = tm.block_prenorm_fwd(x.to(dev), w.to(dev), eps=eps)
    rstd = 1 / torch.sqrt(x.double().square().mean(-1) + eps)
    R.check("rstd", o.rstd, rstd, K * R.U32 * rstd)
    n = x.double() * rstd[:, None] * w.double()
    R.check("n", o.n, n, (half + (K + 2) * R.U32) * n.abs())
    for r in (None, dres):
        b = tm.block_prenorm_bwd(dn.to(dev), x.to(dev), w.to(dev), o.rstd,
                                 dresidual=None if r is None else r.to(dev))
        torch.cuda.synchronize()
        rs = o.rstd.double().cpu()
        dx, dw = R.norm_bwd(dn.double(), x.double(), w.double(), rs)
        mx, mw = R.norm_bwd(dn.double(), x.double(), w.double(), rs, mag=True)
        if r is not None:
            dx, mx = dx + r.double(), mx + r.double().abs()
        R.check("dx", b.dx, dx, half * dx.abs() + (K + 8) * R.U32 * mx)
        R.check("dw", b.dw, dw, half * dw.abs() + (N + 24) * R.U32 * mw)


POST = [  # gate shape as a function of (N, H), post norm, next norm, residual scale
    (lambda N, H: None, True, True, 1.0),
    (lambda N, H: None, False, False, 0.5),
    (lambda N, H: None, False, True, 1.0),
    (lambda N, H: (H,), True, True, 1.0),
    (lambda N, H: (H,), False, False, -2.0),
    (lambda N, H: (N, 1), True, True, 0.25),
    (lambda N, H: (N, 1), False, False, 1.0),
    (lambda N, H: (N, H), True, False, 1.0),
    (lambda N, H: (N // 3, 1, H) if N % 3 == 0 else (1, 1, H), True, True, 1.0),
    (lambda N, H: (3, H) if N % 3 == 0 else (1, H), False, True, 0.0),
    (lambda N, H: (N, H), True, True, 1.0),
    (lambda N, H: (N // 48, H) if N % 48 == 0 else (1, H), True, True, 1.0),
]


def postnorm_case(env, N, H, dt, which, seed=10):
    dev, tm = env
    gate_shape, norm, nxt, scale = POST[which]
    d, half, eps = DT[dt], R.half_step(DT[dt]), 1e-5
    shape = gate_shape(N, H)
    y, res = rnd(seed, N, H, dt=d, scale=0.7), rnd(seed + 1, N, H, dt=d, scale=2.0)
    y[N // 2] = 0
    w = rnd(seed + 2, H, dt=d) + 1 if norm else None
    gate = rnd(seed + 3, *shape, dt=d) if shape else None
    next_w = rnd(seed + 4, H, dt=d) + 1 if nxt else None
    dout, dn = rnd(seed + 5, N, H, dt=d), rnd(seed + 6, N, H, dt=d) if nxt else None
    to = lambda t: None if t is None else t.to(dev)
    K = depth(H)
    o = tm.block_postnorm_fwd(to(y), to(res), to(w), gate=to(gate), next_w=to(next_w),
                              residual_scale=scale, eps=eps)
    torch.cuda.synchronize()
    f = R.postnorm_fwd(y, res, w, gate, next_w, scale, eps)
    e_out = (K + 6) * R.U32 * f["mag"]  # before rounding
    R.check("out", o.out, f["out"], half * f["out"].abs() + e_out)
    if norm:
        R.check("rstd", o.rstd, f["rstd"], K * R.U32 * f["rstd"])
    if nxt:
        # r off by e_out: sum(r^2) by 2 |r| e_out + K 2^-24 r^2, rstd by half that relative
        rel = ((f["out"].abs() * e_out).sum(-1) / H * f["next_rstd"] ** 2 + K * R.U32)
        R.check("next_rstd", o.next_rstd, f["next_rstd"], rel * f["next_rstd"])
        tol = half * f["n"].abs() + (rel[:, None] + 2 * R.U32) * f["n"].abs()
        tol = tol + (e_out * f["next_rstd"][:, None] * next_w.double().abs()) * (1 + half)
        R.check("n", o.n, f["n"], tol)
    b = tm.block_postnorm_bwd(to(dout), to(y), to(w), rstd=o.rstd, gate=to(gate), dn=to(dn),
                              out=o.out, next_w=to(next_w), next_rstd=o.next_rstd,
                              residual_scale=scale)
    torch.cuda.synchronize()
    cpu = lambda t: None if t is None else t.cpu()
    args = (dout, dn, y, o.out.cpu(), w, gate, next_w, cpu(o.rstd), cpu(o.next_rstd), scale)
    ref, mag = R.postnorm_bwd(*args), R.postnorm_bwd(*args, mag=True)
    for name in ("dy", "dresidual", "dw", "dgate", "dnext_w"):
        got = getattr(b, name)
        assert (got is None) == (ref[name] is None), name
        if got is None:
            continue
        # two row sums, then (dw, dgate, dnext_w) a sum over tokens or channels
        chain = 2 * K + 16 + (N if name in ("dw", "dgate", "dnext_w") else 0)
        R.check(name, got, ref[name], half * ref[name].abs() + chain * R.U32 * mag[name])
    return o, b


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("which", range(len(POST)))
@pytest.mark.parametrize("N,H", [(1, 8), (6, 24), (9, 512), (7, 1000), (99, 768), (3, 2056),
                                 (3, 8192), (2, 16384)])
def test_postnorm(env, N, H, which, dt):
    announce(f"postnorm N={N} H={H} case {which} {dt}")
    postnorm_case(env, N, H, dt, which)


@pytest.mark.parametrize("N,H,which", [
    (4200, 40, 3), (4200, 520, 9), (3000, 16, 5), (2049, 64, 0), (60000, 16, 3), (49998, 40, 9),
    (30000, 104, 8), (25001, 200, 0), (9000, 512, 5), (8199, 1000, 9), (3300, 2048, 3),
    (1701, 4096, 9), (900, 6008, 3), (900, 7000, 3), (700, 8200, 5), (700, 16384, 0)])
def test_postnorm_many_rows(env, N, H, which):
    """Units of several rows within a gate's group (or without one), in every layout of threads."""
    announce(f"postnorm N={N} H={H} case {which}")
    postnorm_case(env, N, H, "fp32", which)
    postnorm_case(env, N, H, "bf16", which)


@pytest.mark.parametrize("N,H,which,dt", [
    (60000, 16, 7, "fp32"), (150000, 16, 8, "bf16"), (60000, 104, 7, "bf16"), (30000, 200, 10, "bf16"),
    (9000, 512, 10, "fp32"), (8199, 1000, 8, "bf16"), (8199, 1000, 10, "fp32"),
    (3300, 2048, 8, "bf16"), (1700, 4096, 10, "bf16"), (1700, 3000, 10, "fp32"),
    (900, 6008, 8, "bf16"), (900, 7000, 10, "bf16"), (900, 6008, 7, "bf16"), (900, 6008, 10, "fp32"),
    (700, 16384, 10, "bf16"), (700, 8200, 10, "fp32")])
def test_postnorm_units_of_whole_gate_groups(env, N, H, which, dt):
    """More rows than units, each gate row shared by one token or three: units that hold whole
    groups, in every layout of threads, with and without the next norm."""
    announce(f"postnorm N={N} H={H} case {which} {dt}")
    postnorm_case(env, N, H, dt, which)


@pytest.mark.parametrize("N,H,which", [
    (1200, 200, 8), (600, 768, 8), (4800, 768, 11), (4800, 768, 9), (1536, 4096, 11),
    (768, 16384, 11), (1800, 768, 8), (2304, 1000, 9), (15360, 200, 11), (960, 64, 7),
    (4110, 16, 8), (24960, 1000, 11)])
def test_postnorm_many_gate_rows(env, N, H, which):
    """Gate rows of few units each, and so many that each is a unit of its own."""
    announce(f"postnorm N={N} H={H} case {which}")
    postnorm_case(env, N, H, "fp32", which)
    postnorm_case(env, N, H, "bf16", which)


def test_postnorm_in_place_and_gradient_of_n_alone(env):
    dev, tm = env
    y, res, w = (t.to(dev) for t in (rnd(1, 10, 64), rnd(2, 10, 64), rnd(3, 64)))
    want = tm.block_postnorm_fwd(y, res, w)
    out = res.clone()
    got = tm.block_postnorm_fwd(y, out, w, out=out)
    torch.cuda.synchronize()
    assert got.out.data_ptr() == out.data_ptr() and torch.equal(got.out, want.out)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("which", [i for i, c in enumerate(POST) if c[2]])
@pytest.mark.parametrize("N,H", [(3, 40), (99, 768), (3000, 104), (3, 8200)])
def test_postnorm_gradient_of_n_alone(env, N, H, which, dt):
    """No dout: against the formula, and the bits of a dout of zeros."""
    dev, tm = env
    announce(f"postnorm gradient of n alone N={N} H={H} case {which} {dt}")
    gate_shape, norm, _, scale = POST[which]
    d, half = DT[dt], R.half_step(DT[dt])
    shape = gate_shape(N, H)
    y, res, dn = rnd(1, N, H, dt=d, scale=0.7), rnd(2, N, H, dt=d, scale=2.0), rnd(3, N, H, dt=d)
    w = rnd(4, H, dt=d) + 1 if norm else None
    gate = rnd(5, *shape, dt=d) if shape else None
    next_w = rnd(6, H, dt=d) + 1
    to = lambda t: None if t is None else t.to(dev)
    o = tm.block_postnorm_fwd(to(y), to(res), to(w), gate=to(gate), next_w=to(next_w),
                              residual_scale=scale)
    kw = dict(rstd=o.rstd, gate=to(gate), dn=to(dn), out=o.out, next_w=to(next_w),
              next_rstd=o.next_rstd, residual_scale=scale)
    b = tm.block_postnorm_bwd(None, to(y), to(w), **kw)
    zero = tm.block_postnorm_bwd(torch.zeros(N, H, dtype=d, device=dev), to(y), to(w), **kw)
    torch.cuda.synchronize()
    cpu = lambda t: None if t is None else t.cpu()
    args = (None, dn, y, o.out.cpu(), w, gate, next_w, cpu(o.rstd), cpu(o.next_rstd), scale)
    ref, mag = R.postnorm_bwd(*args), R.postnorm_bwd(*args, mag=True)
    for name in ("dy", "dresidual", "dw", "dgate", "dnext_w"):
        got = getattr(b, name)
        assert (got is None) == (ref[name] is None), name
        if got is None:
            continue
        chain = 2 * depth(H) + 16 + (N if name in ("dw", "dgate", "dnext_w") else 0)
        R.check(name, got, ref[name], half * ref[name].abs() + chain * R.U32 * mag[name])
        assert torch.equal(bits(got), bits(getattr(zero, name))), name


def test_postnorm_bwd_needs_a_gradient(env):
    dev, tm = env
    x, w = torch.zeros(4, 64, device=dev), torch.zeros(64, device=dev)
    with pytest.raises(TypeError):
        tm.block_postnorm_bwd(None, x)
    with pytest.raises(TypeError):
        tm.block_postnorm_bwd(None, x, w, rstd=torch.zeros(4, device=dev))
    with pytest.raises(TypeError):
        tm.block_postnorm_bwd(x, None)
    with pytest.raises(ValueError):
        tm.block_postnorm_bwd(x.cpu(), x)
    side = torch.cuda.Stream()
    b = tm.block_postnorm_bwd(stream=side, y=x, dout=x)
    side.synchronize()
    assert not b.dy.any()


def test_gate_row_per_position_is_refused(env):
    """A gate that torch would broadcast over the batch, not taken for runs of tokens."""
    dev, tm = env
    B, S, H = 2, 4, 64
    y, res, w = rnd(1, B, S, H).to(dev), rnd(2, B, S, H).to(dev), rnd(3, H).to(dev)
    pos = rnd(4, 1, S, H).to(dev)
    o = tm.block_postnorm_fwd(y, res, w)
    for call in (lambda: tm.block_postnorm_fwd(y, res, w, gate=pos),
                 lambda: tm.block_postnorm_bwd(y, y, w, rstd=o.rstd, gate=pos),
                 lambda: tm.block_postnorm(y, res, w, gate=pos),
                 lambda: tm.block_postnorm_fwd(y, res, w, gate=rnd(5, S, B, 1).to(dev))):
        with pytest.raises(ValueError, match="gate"):
            call()
    got = tm.block_postnorm_fwd(y, res, gate=pos.expand(B, S, H).contiguous())
    one = tm.block_postnorm_fwd(y[:1], res[:1], gate=pos)
    torch.cuda.synchronize()
    want = res.double() + pos.double() * y.double()
    mag = (res.abs() + (pos * y).abs()).double().cpu()
    R.check("out", got.out, want.cpu(), 4 * R.U32 * mag)
    assert torch.equal(one.out, got.out[:1])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_token_gate_off_its_allocation(env, dt):
    """The gate of a batch's later tokens: values one by one, at any element's offset."""
    dev, tm = env
    d = DT[dt]
    y, res = rnd(1, 9, 64, dt=d).to(dev), rnd(2, 9, 64, dt=d).to(dev)
    gate, dout = rnd(3, 9, 1, dt=d).to(dev), rnd(4, 9, 64, dt=d).to(dev)
    for first in (1, 2, 3):
        cut = [t[first:] for t in (y, res, gate, dout)]
        o = tm.block_postnorm_fwd(cut[0], cut[1], gate=cut[2])
        want = tm.block_postnorm_fwd(y, res, gate=gate)
        b = tm.block_postnorm_bwd(cut[3], cut[0], gate=cut[2])
        whole = tm.block_postnorm_bwd(dout, y, gate=gate)
        torch.cuda.synchronize()
        assert torch.equal(o.out, want.out[first:])
        for name in ("dy", "dresidual", "dgate"):
            assert torch.equal(getattr(b, name), getattr(whole, name)[first:]), name


def test_norm_infinite_row_stays_in_its_row(env):
    """A row that holds an infinity or NaN gives NaN there and nothing elsewhere."""
    dev, tm = env
    x, w = rnd(1, 9, 72), rnd(2, 72)
    clean = tm.block_prenorm_fwd(x.to(dev), w.to(dev)).n.cpu()
    x[3, 5], x[7, 0] = math.inf, math.nan
    n = tm.block_prenorm_fwd(x.to(dev), w.to(dev)).n.cpu()
    rows = torch.tensor([i for i in range(9) if i not in (3, 7)])
    assert torch.equal(n[rows], clean[rows])
    assert torch.isnan(n[3, 5]) and torch.isnan(n[7]).all()
    assert float(n[3][torch.arange(72) != 5].abs().max()) == 0.0


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_norm_squares_past_the_range(env, dt):
    """A finite row whose squares' sum is infinite in 32 bits: rstd 0, zeros, no gradient of its
    own, and the others' bits as without it."""
    dev, tm = env
    d = DT[dt]
    x, w, dn, dres = rnd(1, 9, 72, dt=d), rnd(2, 72, dt=d), rnd(3, 9, 72, dt=d), rnd(4, 9, 72, dt=d)
    on = [t.to(dev) for t in (x, w, dn, dres)]
    clean = tm.block_prenorm_fwd(on[0], on[1])
    x[3, 5] = 1e20
    on[0] = x.to(dev)
    o = tm.block_prenorm_fwd(on[0], on[1])
    b = tm.block_prenorm_bwd(on[2], on[0], on[1], o.rstd, dresidual=on[3])
    torch.cuda.synchronize()
    others = torch.arange(9) != 3
    assert float(o.rstd[3]) == 0.0 and not o.n[3].any()
    assert torch.equal(o.n.cpu()[others], clean.n.cpu()[others])
    assert torch.equal(b.dx[3], on[3][3]) and bool(b.dw.isfinite().all())


# ------------------------------------------------------------ 8 bits
ACT = [(1, 8), (3, 24), (5, 32), (7, 40), (33, 200), (64, 256), (13, 1000), (100, 2432), (2, 16384)]


def spread(seed, Rn, C, dt):
    """Rows over many magnitudes, zeros, the scale's borders, and values that are not finite."""
    x = rnd(seed, Rn, C)
    x = x * torch.exp2(torch.arange(Rn)[:, None] % 41 * 6.0 - 120)
    x[0, :8] = torch.tensor([448.0, -448.0, 1.0, 0.0, -0.0, 2 ** -9, 2 ** -10, 3 * 2.0 ** -10])
    if Rn > 2:
        x[1, :8] = torch.tensor([449.0, 224.0, 1.75, 0.0, 0.5, 17.0, 19.0, 21.0])
        x[2, :3] = torch.tensor([math.inf, math.nan, -math.inf])
    if Rn > 4:
        x[3] = 0
        x[4, :4] = torch.tensor([3.0e38, -3.0e38, 1e-40, 1e30])
    return x.to(dt)


def check_act8(a, codes, scale):
    got = a.q.view(torch.uint8).cpu().long()
    nan = (codes & 0x7F) == 0x7F
    assert torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], codes[~nan])
    assert torch.equal(a.scale.cpu(), scale)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("Rn,C", ACT)
def test_act8_round_trip(env, Rn, C, dt):
    dev, tm = env
    announce(f"act8 {Rn} x {C} {dt}")
    x = spread(7, Rn, C, DT[dt])
    wide = torch.full((Rn, C + 16), math.nan, dtype=DT[dt])
    wide[:, 8:C + 8] = x
    codes, scale, values = R.act8(x)
    for src in (x.to(dev), wide.to(dev)[:, 8:C + 8]):  # dense, and rows inside wider ones
        a = tm.act8_pack(src)
        torch.cuda.synchronize()
        check_act8(a, codes, scale)
    for out_dt in (torch.float32, torch.bfloat16):
        y = tm.act8_unpack(a.q, a.scale, dtype=out_dt)
        # below the normal numbers a step is 2^-149 (bf16: 2^-133), and half of it the rounding
        tiny = 2.0 ** (-150 if out_dt == torch.float32 else -134)
        R.check("x", y, values, R.half_step(out_dt) * values.abs().nan_to_num() *
                (out_dt != torch.float32) + tiny)
    buf = torch.full((Rn, C + 16), 7.0, dtype=DT[dt], device=dev)
    tm.act8_unpack(a.q, a.scale, x=buf[:, 8:C + 8])
    torch.cuda.synchronize()
    y = tm.act8_unpack(a.q, a.scale, dtype=DT[dt])
    assert torch.equal(bits(buf[:, 8:C + 8].contiguous()), bits(y))
    assert (buf[:, :8] == 7).all() and (buf[:, C + 8:] == 7).all()


def test_act8_every_bf16_value(env):
    """Each bf16 value beside 32 - 1 zeros: the scale rule and the rounding over the whole range."""
    dev, tm = env
    x = torch.zeros(1 << 16, 32, dtype=torch.bfloat16)
    x[:, 3] = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    a = tm.act8_pack(x.to(dev))
    torch.cuda.synchronize()
    codes, scale, _ = R.act8(x)
    check_act8(a, codes, scale)


def test_act8_every_code(env):
    """Every pair of a code and a scale byte back to fp32."""
    dev, tm = env
    q = torch.arange(256, dtype=torch.uint8)[None].expand(255, 256).contiguous()
    s = torch.arange(255, dtype=torch.uint8)[:, None].expand(255, 8).contiguous()
    y = tm.act8_unpack(q.view(torch.float8_e4m3fn).to(dev), s.to(dev), dtype=torch.float32)
    ref = R.from_act8(q, s)
    ref = torch.where(ref.abs() > 3.4028235e38, torch.sign(ref) * math.inf, ref)
    R.check("x", y, ref, torch.full_like(ref, 2.0 ** -150))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("Rn,C", ACT)
@pytest.mark.parametrize("halves", [False, True])
def test_swiglu_act8(env, Rn, C, halves, dt):
    dev, tm = env
    announce(f"swiglu_act8 {Rn} x {C} {dt}")
    d, half = DT[dt], R.half_step(DT[dt])
    gu = rnd(11, Rn, 2 * C, dt=d, scale=3.0)
    gu[0, :6] = torch.tensor([90.0, -90.0, 20.0, -20.0, 0.0, -0.0]).to(d)
    dh = rnd(12, Rn, C, dt=d, scale=0.1)
    on = gu.to(dev)
    g, u = on[:, :C], on[:, C:]
    if not halves:
        g, u = g.contiguous(), u.contiguous()
    o = tm.swiglu_act8_fwd(g, u)
    torch.cuda.synchronize()
    (h, tol), = R.silu_terms(gu[:, :C].double(), gu[:, C:].double())
    R.check("h", o.h, h, half * h.abs() + tol)
    kept = []
    for a, x in ((o.g8, gu[:, :C]), (o.u8, gu[:, C:])):
        codes, scale, v = R.act8(x)
        check_act8(a, codes, scale)
        kept.append(v)
    b = tm.swiglu_act8_bwd(dh.to(dev), o.g8, o.u8)
    torch.cuda.synchronize()
    terms = R.silu_terms(kept[0], kept[1], dh.double())
    for name, (ref, tol) in zip(("h", "dg", "du"), terms):
        R.check(name, getattr(b, name), ref, half * ref.abs() + tol)
    assert b.dg.data_ptr() + C * b.dg.element_size() == b.du.data_ptr()
    dg, du = torch.empty(Rn, C, dtype=d, device=dev), torch.empty(Rn, C, dtype=d, device=dev)
    b2 = tm.swiglu_act8_bwd(dh.to(dev), o.g8, o.u8, with_h=False, dg=dg, du=du)
    torch.cuda.synchronize()
    assert b2.h is None
    assert torch.equal(bits(dg), bits(b.dg.contiguous()))
    assert torch.equal(bits(du), bits(b.du.contiguous()))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_swiglu_act8_far_products(env, dt):
    """g * u past the range of 32 bits where SiLU(g) * u is within it; and of operands
    that 8 bits hold exactly the forward's and the backward's h are the same bits."""
    dev, tm = env
    announce(f"swiglu_act8 products past the range, {dt}")
    d, half = DT[dt], R.half_step(DT[dt])
    g, u = torch.zeros(3, 32), torch.zeros(3, 32)
    g[0], u[0] = -50.0, 1e37
    g[0, 1], u[0, 1] = -40.0, -3e38
    g[1], u[1] = 30.0, 1e37
    g[2], u[2] = -80.0, 1e-3
    g, u = g.to(d), u.to(d)
    o = tm.swiglu_act8_fwd(g.to(dev), u.to(dev))
    (h, tol), = R.silu_terms(g.double(), u.double())
    assert bool(h.isfinite().all())
    R.check("h", o.h, h, half * h.abs() + tol)
    grid = torch.arange(-448, 449, 32, dtype=torch.float32)
    grid = grid[:28].reshape(1, 28) / 64  # multiples of 1/2 up to 7: four bits
    g, u = grid.repeat(2, 1)[:, :24].to(d).to(dev), grid.flip(1).repeat(2, 1)[:, :24].to(d).to(dev)
    o = tm.swiglu_act8_fwd(g, u)
    assert torch.equal(tm.act8_unpack(*o.g8, dtype=d), g)
    b = tm.swiglu_act8_bwd(torch.ones_like(g), o.g8, o.u8)
    torch.cuda.synchronize()
    assert torch.equal(bits(o.h), bits(b.h))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_swiglu_act8_bwd_far_products(env, dt):
    """dh * u past the range of 32 bits where dh * u * SiLU'(g) is within it."""
    dev, tm = env
    announce(f"swiglu_act8 gradients past the range, {dt}")
    d, half = DT[dt], R.half_step(DT[dt])
    g, u, dh = (torch.zeros(3, 32) for _ in range(3))
    g[0], u[0], dh[0] = -50.0, 1e37, 100.0
    g[1], u[1], dh[1] = -30.0, -3e38, 2.0
    g[2], u[2], dh[2] = 20.0, 1e37, 0.5
    g, u, dh = g.to(d), u.to(d), dh.to(d)
    o = tm.swiglu_act8_fwd(g.to(dev), u.to(dev))
    b = tm.swiglu_act8_bwd(dh.to(dev), o.g8, o.u8)
    torch.cuda.synchronize()
    terms = R.silu_terms(R.act8(g)[2], R.act8(u)[2], dh.double())
    for name, (ref, tol) in zip(("h", "dg", "du"), terms):
        assert bool((ref.abs() < 3e38).all())
        R.check(name, getattr(b, name), ref, half * ref.abs() + tol)


def test_swiglu_act8_diverged(env):
    """A value that is not finite is NaN in its own gradients and nowhere else."""
    dev, tm = env
    g, u, dh = rnd(1, 4, 64), rnd(2, 4, 64), rnd(3, 4, 64)
    base = tm.swiglu_act8_fwd(g.to(dev), u.to(dev))
    b0 = tm.swiglu_act8_bwd(dh.to(dev), base.g8, base.u8)
    # (the scale of its group of 32 may change, so that group is left out below)
    g[2, 40] = math.nan
    o = tm.swiglu_act8_fwd(g.to(dev), u.to(dev))
    b = tm.swiglu_act8_bwd(dh.to(dev), o.g8, o.u8)
    torch.cuda.synchronize()
    other = torch.ones(4, 64, dtype=torch.bool)
    other[2, 32:64] = False
    for x, y in ((o.h, base.h), (b.dg, b0.dg), (b.du, b0.du), (b.h, b0.h)):
        assert torch.isnan(x[2, 40])
        assert torch.equal(x.cpu()[other], y.cpu()[other])
        assert not torch.isnan(x[2, 32:40]).any()


# ------------------------------------------------------------ empty, streams, graphs
def test_no_tokens(env):
    dev, tm = env
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=dev)
    o = tm.moe_dispatch_fwd(e(0, 16), e(0, 2, dt=torch.int32), 4)
    assert o.xs.shape == (0, 16) and o.expert_offsets.tolist() == [0] * 5
    assert tm.moe_dispatch_bwd(e(0, 16), o.entry_row).shape == (0, 16)
    assert tm.moe_combine_fwd(e(0, 16), o.entry_row, e(0, 2)).shape == (0, 16)
    c = tm.moe_combine_bwd(e(0, 16), e(0, 16), o.entry_row, e(0, 2))
    assert c.dys.shape == (0, 16) and c.dalpha.shape == (0, 2)
    w = torch.ones(16, device=dev)
    p = tm.block_prenorm_fwd(e(0, 16), w)
    b = tm.block_prenorm_bwd(e(0, 16), e(0, 16), w, p.rstd)
    assert p.n.shape == (0, 16) and b.dw.abs().max() == 0
    for gate in (None, torch.ones(16, device=dev), torch.ones(3, 16, device=dev), e(0, 1), e(0, 16),
                 torch.ones(70000, 16, device=dev)):
        q = tm.block_postnorm_fwd(e(0, 16), e(0, 16), w, gate=gate, next_w=w)
        b = tm.block_postnorm_bwd(e(0, 16), e(0, 16), w, rstd=q.rstd, gate=gate, dn=e(0, 16),
                                  out=q.out, next_w=w, next_rstd=q.next_rstd)
        assert b.dw.abs().max() == 0 and b.dnext_w.abs().max() == 0
        if gate is not None:
            assert b.dgate.shape == gate.shape and not b.dgate.any()
    a = tm.act8_pack(e(0, 40))
    assert a.scale.shape == (0, 2) and tm.act8_unpack(a.q, a.scale).shape == (0, 40)
    s = tm.swiglu_act8_fwd(e(0, 40), e(0, 40))
    assert tm.swiglu_act8_bwd(e(0, 40), s.g8, s.u8).dg.shape == (0, 40)


def block_pass(tm, t, E, cf):
    """One of each, as around a block: outputs in a list."""
    p = tm.block_prenorm_fwd(t["x"], t["w"])
    d = tm.moe_dispatch_fwd(p.n, t["idx"], E, capacity_factor=cf)
    s = tm.swiglu_act8_fwd(d.xs, t["u"])
    y = tm.moe_combine_fwd(s.h, d.entry_row, t["alpha"])
    o = tm.block_postnorm_fwd(y, t["x"], t["w"], gate=t["gate"], next_w=t["w2"])
    b = tm.block_postnorm_bwd(t["dout"], y, t["w"], rstd=o.rstd, gate=t["gate"], dn=t["dn"],
                              out=o.out, next_w=t["w2"], next_rstd=o.next_rstd)
    c = tm.moe_combine_bwd(b.dy, s.h, d.entry_row, t["alpha"])
    g = tm.swiglu_act8_bwd(c.dys, s.g8, s.u8)
    a = tm.act8_pack(g.dg)
    dxs = tm.act8_unpack(a.q, a.scale, dtype=t["x"].dtype)
    dn = tm.moe_dispatch_bwd(dxs, d.entry_row)
    f = tm.block_prenorm_bwd(dn, t["x"], t["w"], p.rstd, dresidual=b.dresidual)
    return [p.n, d.xs, d.entry_row, s.h, s.g8.q.view(torch.uint8), y, o.out, o.n, b.dw, b.dgate,
            b.dnext_w, c.dalpha, g.du, g.h, f.dx, f.dw]


def block_inputs(dev, seed, N, H, E, k, dt):
    d = DT[dt]
    t = {"x": rnd(seed, N, H, dt=d), "w": rnd(seed + 1, H, dt=d), "w2": rnd(seed + 2, H, dt=d),
         "gate": rnd(seed + 3, H, dt=d), "u": rnd(seed + 4, N * k, H, dt=d),
         "dout": rnd(seed + 5, N, H, dt=d), "dn": rnd(seed + 6, N, H, dt=d),
         "alpha": torch.rand(N, k, generator=torch.Generator().manual_seed(seed)),
         "idx": route(seed, N, E, k, 0.1, False)}
    return {n: v.to(dev) for n, v in t.items()}


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b))


@pytest.mark.parametrize("N,H,E,k,dt", [(32, 256, 8, 2, "bf16"), (1500, 104, 16, 2, "fp32"),
                                           (16500, 40, 16, 2, "bf16")])
def test_deterministic_streams_and_graph(env, N, H, E, k, dt):
    dev, tm = env
    announce(f"block pass N={N} H={H} {dt}: again, another stream, captured")
    t = block_inputs(dev, 40, N, H, E, k, dt)
    t2 = block_inputs(dev, 60, N, H, E, k, dt)
    want = block_pass(tm, t, E, 1.0)
    torch.cuda.synchronize()
    assert same(want, block_pass(tm, t, E, 1.0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block_pass(tm, t, E, 1.0)
    side.synchronize()
    assert same(want, got)
    # the stream argument alone, as an object and as a raw handle
    for s in (side, side.cuda_stream):
        p = tm.block_prenorm_fwd(t["x"], t["w"], stream=s)
        side.synchronize()
        assert same([p.n], want[:1])
    want2 = block_pass(tm, t2, E, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block_pass(tm, t, E, 1.0)
    keep = {n: v.clone() for n, v in t.items()}
    for r in range(4):
        for n in t:  # new inputs in the captured buffers on every second replay
            t[n].copy_(t2[n] if r % 2 else keep[n])
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, want2 if r % 2 else want), r
        assert same(block_pass(tm, t2, E, 1.0), want2)  # eager work between the replays
        torch.randn(1 << 16, device=dev).sum().item()


def test_two_streams_at_once(env):
    """Two passes of different inputs in flight at the same time."""
    dev, tm = env
    a, b = (block_inputs(dev, seed, 16500, 104, 16, 2, "bf16") for seed in (40, 60))
    want = [block_pass(tm, t, 16, 1.0) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in want]
    for turn in range(3):
        got = []
        for t, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append(block_pass(tm, t, 16, 1.0))
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(got, want)), turn


@pytest.mark.parametrize("N,H,G", [(20000, 64, 1), (100, 768, 4), (4096, 64, 4096)])
def test_buffers_of_the_caller(env, N, H, G):
    """Workspaces and outputs given, with other bytes in them, one workspace for calls in turn."""
    dev, tm = env
    announce(f"given buffers N={N} H={H} gate rows {G}")
    E, k = 8, 2
    x, dn, y = (rnd(i, N, H).to(dev) for i in range(3))
    w, gate, idx = rnd(3, H).to(dev), rnd(4, G, H).to(dev), route(5, N, E, k, 0.1, False).to(dev)
    nan = lambda *s: torch.full(s, math.nan, device=dev)
    size = max(tm.moe_dispatch_workspace_bytes(N, E, k), tm.block_norm_bwd_workspace_bytes(N, H),
               tm.block_norm_bwd_workspace_bytes(N, H, G))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=dev)
    d = tm.moe_dispatch_fwd(x, idx, E, xs=nan(N * k, H), workspace=ws)
    p = tm.block_prenorm_fwd(x, w, n=nan(N, H))
    b = tm.block_prenorm_bwd(dn, x, w, p.rstd, workspace=ws)
    o = tm.block_postnorm_fwd(y, x, w, gate=gate, next_w=w, out=nan(N, H))
    kw = dict(rstd=o.rstd, gate=gate, dn=dn, out=o.out, next_w=w, next_rstd=o.next_rstd)
    q = tm.block_postnorm_bwd(dn, y, w, workspace=ws, **kw)
    back = tm.moe_dispatch_bwd(d.xs, d.entry_row, dx=nan(N, H))
    alpha = torch.rand(N, k, device=dev)
    c = tm.moe_combine_fwd(d.xs, d.entry_row, alpha, y=nan(N, H))
    torch.cuda.synchronize()
    got = [*d, *p, *b, *o, *q, back, c]
    d = tm.moe_dispatch_fwd(x, idx, E)
    p = tm.block_prenorm_fwd(x, w)
    o = tm.block_postnorm_fwd(y, x, w, gate=gate, next_w=w)
    want = [*d, *p, *tm.block_prenorm_bwd(dn, x, w, p.rstd), *o, *tm.block_postnorm_bwd(dn, y, w, **kw),
            tm.moe_dispatch_bwd(d.xs, d.entry_row), tm.moe_combine_fwd(d.xs, d.entry_row, alpha)]
    torch.cuda.synchronize()
    assert same(got, want)


def test_gpu_refusals(env):
    """Calls that the front end or the library turns down before anything is launched."""
    dev, tm = env
    from top_moe_layer_amd import TopmoeError

    x, w = torch.zeros(4, 64, device=dev), torch.zeros(64, device=dev)
    idx = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    odd = torch.zeros(4 * 64 + 1, device=dev)[1:].view(4, 64)  # 4 bytes off its allocation
    g8 = tm.act8_pack(x)
    bad = [
        (ValueError, lambda: tm.block_prenorm_fwd(x.t(), torch.zeros(4, device=dev))),
        (ValueError, lambda: tm.block_prenorm_fwd(x, w[:32])),
        (TypeError, lambda: tm.block_prenorm_fwd(x, w.to(torch.bfloat16))),
        (TypeError, lambda: tm.block_prenorm_fwd(x.half(), w.half())),
        (ValueError, lambda: tm.block_prenorm_fwd(x, w.cpu())),
        (TopmoeError, lambda: tm.block_prenorm_fwd(odd, w)),
        (TopmoeError, lambda: tm.block_prenorm_fwd(x, w, eps=0.0)),
        (TopmoeError, lambda: tm.block_prenorm_fwd(x[:, :60].contiguous(), w[:60].contiguous())),
        (ValueError, lambda: tm.block_postnorm_fwd(x, x, gate=torch.zeros(3, 64, device=dev))),
        (ValueError, lambda: tm.block_postnorm_fwd(x, x, gate=torch.zeros(4, device=dev))),
        (ValueError, lambda: tm.block_postnorm_fwd(x, x[:2])),
        (ValueError, lambda: tm.block_postnorm_bwd(x, x, dn=x)),
        (TypeError, lambda: tm.block_postnorm_bwd(x, x, w)),  # no rstd
        (ValueError, lambda: tm.block_prenorm_bwd(x, x, w, torch.zeros(4, device=dev),
                                                  workspace=torch.zeros(8, device=dev))),
        (TypeError, lambda: tm.moe_dispatch_fwd(x, idx.long(), 4)),
        (ValueError, lambda: tm.moe_dispatch_fwd(x, idx[:2], 4)),
        (ValueError, lambda: tm.moe_dispatch_fwd(x, idx[:, 0], 4)),
        (TopmoeError, lambda: tm.moe_dispatch_fwd(x, idx, 0)),
        (TopmoeError, lambda: tm.moe_dispatch_fwd(x, idx, 10 ** 12)),
        (TopmoeError, lambda: tm.moe_dispatch_fwd(x, idx, 1)),  # k > E
        (TopmoeError, lambda: tm.moe_dispatch_fwd(x, idx, 4, capacity_factor=-1.0)),
        (TopmoeError, lambda: tm.moe_dispatch_fwd(odd, idx, 4)),
        (ValueError, lambda: tm.moe_combine_fwd(x, idx, torch.zeros(4, 2, device=dev))),  # 8 rows
        (TypeError, lambda: tm.moe_combine_fwd(torch.zeros(8, 64, device=dev), idx,
                                               torch.zeros(4, 2, device=dev).half())),
        (ValueError, lambda: tm.act8_pack(x.t())),
        (ValueError, lambda: tm.act8_pack(x.view(2, 2, 64))),
        (ValueError, lambda: tm.act8_pack(x[:1].expand(4, 64))),
        (TopmoeError, lambda: tm.act8_pack(x[:, :60])),
        (TopmoeError, lambda: tm.act8_pack(x[:, 2:34])),  # rows that begin off 16 bytes
        (ValueError, lambda: tm.act8_unpack(g8.q, g8.scale[:, :1])),
        (TypeError, lambda: tm.act8_unpack(g8.q.view(torch.uint8), g8.scale)),
        (ValueError, lambda: tm.swiglu_act8_bwd(x, g8, g8, dg=x)),
        (TopmoeError, lambda: tm.ffn_swiglu_keep8(x, 4, 64, 64, torch.float32)),  # too small
        (TopmoeError, lambda: tm.ffn_swiglu_keep8(x, 4, 64, 60, torch.float32)),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(f"call {i} was taken")
    torch.cuda.synchronize()


def test_stage_events(env):
    dev, tm = env
    for N in (16, 40000):  # one launch, three launches
        x, idx = rnd(1, N, 64).to(dev), route(1, N, 4, 1, 0.0, False).to(dev)
        ev = tm.StageEvents(tm.DISPATCH_STAGES)
        o = tm.moe_dispatch_fwd(x, idx, 4, stage_events=ev)
        assert all(v >= 0 for v in ev.elapsed_ms())
        plain = tm.moe_dispatch_fwd(x, idx, 4)
        assert torch.equal(o.xs, plain.xs)
    w = torch.ones(64, device=dev)
    p = tm.block_prenorm_fwd(x, w)
    ev = tm.StageEvents(tm.NORM_BWD_STAGES)
    tm.block_prenorm_bwd(x, x, w, p.rstd, stage_events=ev)
    assert all(v > 0 for v in ev.elapsed_ms())


def test_stage_events_of_another_call(env):
    """Events for fewer stages than the call has are refused."""
    dev, tm = env
    x, w = rnd(1, 16, 64).to(dev), torch.ones(64, device=dev)
    idx = route(1, 16, 4, 1, 0.0, False).to(dev)
    p = tm.block_prenorm_fwd(x, w)
    with pytest.raises(ValueError, match="stages"):
        tm.block_prenorm_bwd(x, x, w, p.rstd, stage_events=tm.StageEvents(1))
    with pytest.raises(ValueError, match="stages"):
        tm.moe_dispatch_fwd(x, idx, 4, stage_events=tm.StageEvents(1))
    one = tm.StageEvents(1)
    tm.block_prenorm_fwd(x, w, stage_events=one)
    assert one.elapsed_ms()[0] > 0
