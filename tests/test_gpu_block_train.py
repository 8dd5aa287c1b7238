"""The block operators inside a PyTorch graph, together as a block with experts
of the caller's own uses them, and the FFN / MoE training path with g and u
kept in 8 bits between the passes."""
import numpy as np
import pytest
import torch

import block_ref as R
from gpu_util import TOL_GRAD, announce, rel_l2_per_matrix, rel_l2_per_token, torch_dev

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


def eq(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------ one Function each
def test_functions_are_their_entry_points(env):
    """Each Function's outputs and gradients are the bits of its forward and backward."""
    dev, tm = env
    B, S, H, E, k = 3, 20, 72, 5, 2
    N = B * S
    leaf = lambda t: t.to(dev).requires_grad_()
    x, w = leaf(rnd(1, B, S, H)), leaf(rnd(2, H))
    n = tm.block_prenorm(x, w, 1e-4)
    dn = rnd(3, B, S, H).to(dev)
    n.backward(dn)
    o = tm.block_prenorm_fwd(x.detach(), w.detach(), eps=1e-4)
    g = tm.block_prenorm_bwd(dn, x.detach(), w.detach(), o.rstd)
    assert eq(n, o.n) and eq(x.grad, g.dx) and eq(w.grad, g.dw)

    y, res, gate, w2 = leaf(rnd(4, B, S, H)), leaf(rnd(5, B, S, H)), leaf(rnd(6, B, 1, H)), leaf(rnd(7, H))
    w = leaf(rnd(2, H))
    dout = rnd(8, B, S, H).to(dev)
    for use in ("both", "out", "n"):
        for t in (y, res, gate, w, w2):
            t.grad = None
        out, n = tm.block_postnorm(y, res, w, gate=gate, next_w=w2, residual_scale=0.5)
        loss = {"both": (out * dout).sum() + (n * dn).sum(), "out": (out * dout).sum(),
                "n": (n * dn).sum()}[use]
        loss.backward()
        d = [t.detach() for t in (y, res, w, gate, w2)]
        o = tm.block_postnorm_fwd(d[0], d[1], d[2], gate=d[3], next_w=d[4], residual_scale=0.5)
        kw = {} if use == "out" else dict(dn=dn, out=o.out, next_w=d[4], next_rstd=o.next_rstd)
        g = tm.block_postnorm_bwd(torch.zeros_like(dout) if use == "n" else dout, d[0], d[2],
                                  rstd=o.rstd, gate=d[3], residual_scale=0.5, **kw)
        assert eq(out, o.out) and eq(n, o.n)
        assert eq(y.grad, g.dy) and eq(res.grad, g.dresidual) and eq(w.grad, g.dw)
        assert eq(gate.grad, g.dgate)
        assert w2.grad is None if use == "out" else eq(w2.grad, g.dnext_w)
    out = tm.block_postnorm(y, res)
    assert torch.equal(out, y + res)

    x = leaf(rnd(9, B, S, H))
    idx = torch.randint(-1, E, (N, k), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    alpha = leaf(torch.rand(N, k))
    r = tm.moe_dispatch(x, idx.to(dev), E, capacity_factor=1.0)
    res = leaf(rnd(10, N, H))
    y = tm.moe_combine(r.xs, r.entry_row, alpha, res)
    dy = rnd(11, N, H).to(dev)
    y.backward(dy)
    c = tm.moe_combine_bwd(dy, r.xs.detach(), r.entry_row, alpha.detach())
    assert eq(alpha.grad, c.dalpha) and eq(res.grad, dy)
    assert eq(x.grad, tm.moe_dispatch_bwd(c.dys, r.entry_row).view(B, S, H))

    C = 40
    gu = leaf(rnd(12, B, S, 2 * C))
    h = tm.swiglu_act8(gu)
    dh = rnd(13, B, S, C).to(dev)
    h.backward(dh)
    flat = gu.detach().view(N, 2 * C)
    o = tm.swiglu_act8_fwd(flat[:, :C], flat[:, C:])
    b = tm.swiglu_act8_bwd(dh.view(N, C), o.g8, o.u8)
    assert eq(h.view(N, C), o.h) and eq(gu.grad.view(N, 2 * C), torch.cat([b.dg, b.du], 1))
    g1, u1 = leaf(gu.detach()[..., :C].cpu()), leaf(gu.detach()[..., C:].cpu())
    tm.swiglu_act8(g1, u1).backward(dh)
    assert eq(g1.grad.view(N, C), b.dg) and eq(u1.grad.view(N, C), b.du)
    with pytest.raises(ValueError):
        tm.swiglu_act8(rnd(1, 4, 7).to(dev))


def test_swiglu_act8_operands_of_one_shape(env):
    """As many values in another shape are not an operand."""
    dev, tm = env
    g = rnd(1, 2, 3, 64).to(dev)
    for u in (rnd(2, 3, 2, 64), rnd(2, 6, 64), rnd(2, 2, 6, 32)):
        with pytest.raises(ValueError, match="shape"):
            tm.swiglu_act8(g, u.to(dev))
    assert tm.swiglu_act8(g, rnd(2, 2, 3, 64).to(dev)).shape == g.shape


def test_postnorm_gradient_of_n_alone_takes_no_zeros(env):
    """A loss of n alone: no tensor of zeros is made for the gradient of out."""
    dev, tm = env
    N, H = 4096, 512
    y, res, w = (t.to(dev).requires_grad_() for t in (rnd(1, N, H), rnd(2, N, H), 1 + rnd(3, H)))
    dn = rnd(4, N, H).to(dev)
    n = tm.block_postnorm(y, res, w, next_w=w)[1]
    for t in (y, res, w):
        t.grad = torch.zeros_like(t)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    n.backward(dn)
    torch.cuda.synchronize()
    # dy, dresidual and the partial sums (2 * 2048 units * H floats, once more as much as a
    # tensor of the rows), but no third tensor of the rows beside the small ones
    rows, sums = N * H * 4, tm.block_norm_bwd_workspace_bytes(N, H)
    assert torch.cuda.max_memory_allocated() - before < 2.9 * rows + sums


def functions(dev, tm, dt):
    """Every Function with its leaves: name -> (leaves, call)."""
    N, H, I, E, k = 40, 64, 64, 4, 2
    d = DT[dt]
    leaf = lambda seed, *s, t=d, scale=0.5: rnd(seed, *s, dt=t, scale=scale).to(dev).requires_grad_()
    idx = torch.randint(-1, E, (N, k), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    idx = idx.to(dev)
    er = tm.moe_dispatch_fwd(torch.zeros(N, H, dtype=d, device=dev), idx, E).entry_row
    x, w, f32 = leaf(1, N, H), leaf(2, H), torch.float32
    ffn = [leaf(3, I, H), leaf(4, I, H), leaf(5, H, I)]
    moe = [leaf(6, E, H, t=f32), leaf(7, E, I, H), leaf(8, E, I, H), leaf(9, E, H, I)]
    ys, alpha, w2, gate = leaf(10, N * k, H), leaf(11, N, k, t=f32), leaf(12, H), leaf(13, H)
    out = {
        "prenorm": ([x, w], lambda: tm.block_prenorm(x, w)),
        "postnorm": ([x, w, gate], lambda: tm.block_postnorm(x, x, w, gate=gate)),
        "postnorm n": ([x, w, w2], lambda: tm.block_postnorm(x, x, w, next_w=w2)[1]),
        "dispatch": ([x], lambda: tm.moe_dispatch(x, idx, E).xs),
        "combine": ([ys, alpha, x], lambda: tm.moe_combine(ys, er, alpha, x)),
        "swiglu": ([ys], lambda: tm.swiglu_act8(ys)),
    }
    for keep in (False, True, "act8"):
        out[f"ffn {keep}"] = ([x, *ffn], lambda keep=keep: tm.swiglu_ffn(x, *ffn, x, keep_activations=keep))
        out[f"moe {keep}"] = ([x, *moe], lambda keep=keep: tm.moe_ffn(x, *moe, k, 0.0, keep_activations=keep)[0])
    return out


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_upstream_gradients_at_any_offset(env, dt):
    """The gradient of a piece of a concatenation begins at any element, that of a sum is expanded
    from one value: both as a tensor of their own."""
    dev, tm = env
    one = torch.ones(1, dtype=DT[dt], device=dev)
    for name, (leaves, call) in functions(dev, tm, dt).items():
        announce(f"gradient at an odd offset: {name} {dt}")
        y = call()
        dy = rnd(20, *y.shape, dt=DT[dt]).to(dev)
        want = torch.autograd.grad(y, leaves, dy)
        y = call()
        cat = torch.cat([one, y.flatten()])
        got = torch.autograd.grad(cat, leaves, torch.cat([one, dy.flatten()]))
        assert all(eq(a, b) for a, b in zip(got, want)), name
        want = torch.autograd.grad(call(), leaves, torch.ones_like(dy))
        got = torch.autograd.grad(call().sum(), leaves)
        assert all(eq(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_functions_captured(env, dt):
    """Forward and backward of every Function in one graph, replayed over new inputs."""
    dev, tm = env
    fs = functions(dev, tm, dt)
    leaves = list({id(t): t for l, _ in fs.values() for t in l}.values())
    ups = {n: rnd(30, *call().shape, dt=DT[dt]).to(dev) for n, (_, call) in fs.items()}

    def step():
        res = []
        for name, (l, call) in fs.items():
            y = call()
            # (a residual's gradient is the upstream gradient itself, which is cleared below)
            res += [t.clone() for t in (y.detach(), *torch.autograd.grad(y, l, ups[name]))]
        return res

    first = [t.detach().clone() for t in leaves]
    second = [torch.randn_like(t) * 0.5 for t in first]
    want = {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.no_grad():
        for name, src in (("2", second), ("1", first)):
            for t, v in zip(leaves, src):
                t.copy_(v)
            with torch.enable_grad():
                want[name] = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for r in range(4):
        name, src = ("1", first) if r % 2 == 0 else ("2", second)
        with torch.no_grad():
            for t, v in zip(leaves, src):
                t.copy_(v)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(eq(a, b) for a, b in zip(outs, want[name])), r
        assert all(eq(a, b) for a, b in zip(step(), want[name]))  # eager work between the replays


# ------------------------------------------------------------ a block of its own experts
def block_forward(P, k, E, cf, ops, act8):
    """One pre- and post-normed MoE block whose experts are the caller's own
    products; `ops` the library or its plain form."""
    x = P["x"]
    n = ops.prenorm(x, P["w1"])
    p = torch.softmax(n @ P["Wr"].T, -1)
    alpha, idx = torch.topk(p, k, dim=-1)
    alpha = alpha / alpha.sum(-1, keepdim=True)
    xs, off, entry_row = ops.dispatch(n, idx.to(torch.int32), E, cf)
    ys = []
    for e in range(E):
        rows = xs[off[e]:off[e + 1]]
        gu = rows @ P["Wgu"][e].T
        ys.append(ops.swiglu(gu, act8) @ P["Wd"][e].T)
    ys.append(0.0 * xs[off[E]:])
    y = ops.combine(torch.cat(ys), entry_row, alpha)
    out, n2 = ops.postnorm(y, x, P["w2"], P["gate"], P["w3"])
    return out, n2


class Lib:
    def __init__(self, tm):
        self.tm = tm

    def prenorm(self, x, w):
        return self.tm.block_prenorm(x, w)

    def dispatch(self, n, idx, E, cf):
        r = self.tm.moe_dispatch(n, idx.contiguous(), E, capacity_factor=cf)
        return r.xs, r.expert_offsets.tolist(), r.entry_row

    def swiglu(self, gu, act8):
        if act8:
            return self.tm.swiglu_act8(gu)
        g, u = gu.chunk(2, -1)
        return torch.nn.functional.silu(g) * u

    def combine(self, ys, entry_row, alpha):
        return self.tm.moe_combine(ys, entry_row, alpha.float())

    def postnorm(self, y, x, w, gate, w3):
        return self.tm.block_postnorm(y, x, w, gate=gate, next_w=w3, residual_scale=0.8)


class Plain:
    """The same in elementary differentiable operations."""

    def prenorm(self, x, w):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w

    def dispatch(self, n, idx, E, cf):
        N, k = idx.shape
        off, row_entry, entry_row = R.rows_of(idx.tolist(), E, cf)
        at = torch.tensor([max(i, 0) for i in row_entry]) // k
        keep = torch.tensor([float(i >= 0) for i in row_entry], dtype=n.dtype)
        return n[at] * keep[:, None], off, torch.tensor(entry_row).reshape(N, k)

    def swiglu(self, gu, act8):
        g, u = gu.chunk(2, -1)
        return g * torch.sigmoid(g) * u

    def combine(self, ys, entry_row, alpha):
        keep = (entry_row >= 0).to(ys.dtype)
        return (ys[entry_row.clamp(min=0)] * (alpha * keep)[..., None]).sum(1)

    def postnorm(self, y, x, w, gate, w3):
        out = 0.8 * x + gate * self.prenorm(y, w)
        return out, self.prenorm(out, w3)


@pytest.mark.parametrize("cf", [0.0, 0.75])
@pytest.mark.parametrize("act8", [False, True])
def test_block_with_own_experts(env, act8, cf):
    """Outputs and every gradient of a block, fp32, against 64 bits.  The
    longest chain of dependent sums is about 2 H + 2 I + 64 = 500 roundings of
    2^-24; norms, routing weights and SwiGLU pass an error on at most about
    eightfold each (|x| / rms and |g| stay below 8 here): 500 * 2^-24 * 32 =
    1e-3 of an output's norm.  With g and u in 8 bits each gradient term is off
    by at most 3 * 2^-4 of itself (g, u and silu'(g) each by half a step)."""
    dev, tm = env
    announce(f"block with own experts, act8={act8}, capacity factor {cf}")
    N, H, I, E, k = 93, 64, 96, 4, 2
    P = {"x": rnd(1, N, H), "w1": 1 + 0.1 * rnd(2, H), "Wr": rnd(3, E, H) * 0.3,
         "Wgu": rnd(4, E, 2 * I, H) * H ** -0.5, "Wd": rnd(5, E, H, I) * I ** -0.5,
         "w2": 1 + 0.1 * rnd(6, H), "gate": 0.5 + 0.1 * rnd(7, H), "w3": 1 + 0.1 * rnd(8, H)}
    d1, d2 = rnd(9, N, H), rnd(10, N, H)
    A = {n: t.double().requires_grad_() for n, t in P.items()}
    B = {n: t.to(dev).requires_grad_() for n, t in P.items()}
    ref = block_forward(A, k, E, cf, Plain(), act8)
    ((ref[0] * d1).sum() + (ref[1] * d2).sum()).backward()
    got = block_forward(B, k, E, cf, Lib(tm), act8)
    ((got[0] * d1.to(dev)).sum() + (got[1] * d2.to(dev)).sum()).backward()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert float((b.detach().double().cpu() - a.detach()).norm() / a.detach().norm()) <= 1e-3
    for n in P:
        a, b = A[n].grad, B[n].grad.double().cpu()
        assert float((b - a).norm() / a.norm()) <= (3 / 16 if act8 else 1e-3), n


# ------------------------------------------------------------ the FFN's own g, u in 8 bits
def parts(kept, start, rows, I):
    """g and u (float64) from the bytes of a kept buffer whose 8-bit parts begin at `start`."""
    up = lambda v: -(-v // 256) * 256
    b = kept.cpu()
    n = rows * I
    at = [up(start)]
    for size in (n, n, n // 32):
        at.append(up(at[-1] + size))
    gq, uq = (b[a:a + n].reshape(rows, I) for a in at[:2])
    gs, us = (b[a:a + n // 32].reshape(rows, I // 32) for a in at[2:])
    return (R.from_act8(gq, gs), gs), (R.from_act8(uq, us), us)


def check_kept(v, scale, exact, dt):
    """8-bit values of an activation computed by the GEMM: half a step of e4m3
    (2^-4 relative, or 2^-10 of the scale below its normal numbers) of the
    value rounded to the dtype, itself within 2^-7 (bf16) / 2^-12 (fp32, a sum
    of H terms in 32 bits) of the exact product's magnitude here."""
    step = torch.exp2(scale.double() - 127 - 10).repeat_interleave(32, 1)
    near = 2.0 ** (-7 if dt == "bf16" else -12)
    tol = (2.0 ** -4 + near) * exact.abs() + step + near * exact.abs().mean()
    assert bool(((v - exact).abs() <= tol).all())


def swiglu_grads(g, u, dh):
    s = torch.sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s, g * s * u


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,I", [(1, 64, 64), (130, 128, 192), (300, 256, 704)])
def test_dense_keep8(env, N, H, I, dt):
    dev, tm = env
    announce(f"dense keep8 N={N} H={H} I={I} {dt}")
    d = DT[dt]
    x, dy = rnd(1, N, H, dt=d), rnd(2, N, H, dt=d)
    Wg, Wu, Wd = rnd(3, I, H, dt=d, scale=H ** -0.5), rnd(4, I, H, dt=d, scale=H ** -0.5), \
        rnd(5, H, I, dt=d, scale=I ** -0.5)
    D = [t.to(dev) for t in (x, Wg, Wu, Wd)]
    saved = torch.empty(tm.ffn_bwd_workspace_bytes(N, H, I, d), dtype=torch.uint8, device=dev)
    y = tm.ffn_swiglu_fwd(*D, saved=saved)
    kept = tm.ffn_swiglu_keep8(saved, N, H, I, d)
    assert kept.numel() == tm.ffn_keep8_bytes(N, H, I, d)
    saved.fill_(255)  # NaN in every type: nothing may be read from it again
    ws = tm.ffn_swiglu_restore8(kept, N, H, I, d, workspace=saved)
    out = tm.ffn_swiglu_bwd(*D, dy.to(dev), workspace=ws, from_saved=True)
    torch.cuda.synchronize()
    X, DY, WG, WU, WD = (t.double() for t in (x, dy, Wg, Wu, Wd))
    (g, gs), (u, us) = parts(kept, 0, N, I)
    check_kept(g, gs, X @ WG.T, dt)
    check_kept(u, us, X @ WU.T, dt)
    dg, du, h = swiglu_grads(g, u, DY @ WD)
    np_ = lambda t: t.double().cpu().numpy()
    assert rel_l2_per_token(np_(out.dx), np_(dg @ WG + du @ WU)) <= TOL_GRAD[dt]
    for got, ref in ((out.dWg, dg.T @ X), (out.dWu, du.T @ X), (out.dWd, DY.T @ h)):
        assert rel_l2_per_matrix(np_(got), np_(ref)) <= TOL_GRAD[dt]

    # inside autograd: y's bits without it, these gradients' bits, twice over one graph
    L = [t.clone().requires_grad_() for t in D]
    ya = tm.swiglu_ffn(*L, keep_activations="act8")
    for _ in range(2):
        for t in L:
            t.grad = None
        ya.backward(dy.to(dev), retain_graph=True)
        assert eq(ya, y)
        for t, ref in zip(L, (out.dx, out.dWg, out.dWu, out.dWd)):
            assert eq(t.grad, ref)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H,I,E,k,cf", [(5, 64, 64, 4, 2, 0.0), (200, 128, 192, 8, 2, 0.0),
                                          (333, 64, 128, 3, 1, 0.6), (150, 64, 64, 6, 3, 0.5)])
def test_moe_keep8(env, N, H, I, E, k, cf, dt):
    dev, tm = env
    announce(f"MoE keep8 N={N} H={H} I={I} E={E} k={k} cf={cf} {dt}")
    d = DT[dt]
    x, dy, Wr = rnd(1, N, H, dt=d), rnd(2, N, H, dt=d), rnd(6, E, H, scale=H ** -0.5)
    Wg, Wu, Wd = rnd(3, E, I, H, dt=d, scale=H ** -0.5), rnd(4, E, I, H, dt=d, scale=H ** -0.5), \
        rnd(5, E, H, I, dt=d, scale=I ** -0.5)
    D = [t.to(dev) for t in (x, Wr, Wg, Wu, Wd)]
    kw = dict(norm_topk_prob=False, capacity_factor=cf)
    saved = torch.empty(tm.moe_bwd_workspace_bytes(N, H, I, E, k, d), dtype=torch.uint8, device=dev)
    o = tm.moe_ffn_fwd(*D, k, 0.0, saved=saved, **kw)
    kept = tm.moe_ffn_keep8(saved, N, H, I, E, k, d)
    assert kept.numel() == tm.moe_keep8_bytes(N, H, I, E, k, d)
    saved.fill_(255)
    ws = tm.moe_ffn_restore8(kept, N, H, I, E, k, d, workspace=saved)
    out = tm.moe_ffn_bwd(*D, dy.to(dev), k, 0.0, workspace=ws, from_saved=True, **kw)
    torch.cuda.synchronize()
    X, DY, WR, WG, WU, WD = (t.double() for t in (x, dy, Wr, Wg, Wu, Wd))
    rows = N * k
    up = lambda v: -(-v // 256) * 256
    n = rows * I  # g, u, their scales (the last part ends the buffer)
    start = kept.numel() - 2 * up(n) - up(n // 32) - up(n // 32 + 1)
    (g, gs), (u, us) = parts(kept, start, rows, I)
    p = torch.softmax(X @ WR.T, -1)
    idx, off = o.topk_idx.cpu().long(), o.expert_offsets.tolist()
    tok = o.sorted_token_ids.cpu().long()
    dx = torch.zeros(N, H, dtype=torch.float64)
    dWg, dWu, dWd = (torch.zeros_like(t) for t in (WG, WU, WD))
    dp = torch.zeros(N, E, dtype=torch.float64)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        t = tok[r]
        if not len(t):
            continue
        check_kept(g[r], gs[r], X[t] @ WG[e].T, dt)
        check_kept(u[r], us[r], X[t] @ WU[e].T, dt)
        raw = DY[t] @ WD[e]
        a = p[t, e][:, None]
        dg, du, h = swiglu_grads(g[r], u[r], a * raw)
        dx.index_add_(0, t, dg @ WG[e] + du @ WU[e])
        dWg[e], dWu[e], dWd[e] = dg.T @ X[t], du.T @ X[t], (a * DY[t]).T @ h
        dp[t, e] = (raw * h).sum(-1)
    assert (idx >= 0).all()
    dr = p * (dp - (p * dp).sum(-1, keepdim=True))
    dx += dr @ WR
    np_ = lambda t: t.double().cpu().numpy()
    live = dx.norm(dim=1) > 0  # a token all of whose entries were dropped
    assert rel_l2_per_matrix(np_(out.dx), np_(dx)) <= TOL_GRAD[dt]
    assert bool(live.any())
    for n, ref in (("dWg", dWg), ("dWu", dWu), ("dWd", dWd)):
        assert rel_l2_per_matrix(np_(getattr(out, n)), np_(ref)) <= TOL_GRAD[dt], n
    assert rel_l2_per_matrix(np_(out.dWr), np_(dr.T @ X)) <= TOL_GRAD[dt]

    L = [t.clone().requires_grad_() for t in D]
    ya = tm.moe_ffn(*L, k, 0.0, keep_activations="act8", **kw)[0]
    ya.backward(dy.to(dev))
    assert eq(ya, o.y)
    for t, ref in zip(L, (out.dx, out.dWr, out.dWg, out.dWu, out.dWd)):
        assert eq(t.grad, ref)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_keep8_products_next_to_the_range(env, dt):
    """g * u within the range of 32 bits before they are kept and past it as kept (-59 and 1.07 *
    2^122 as -60 and 1.125 * 2^122), SiLU(g) * u far within: the down weights' gradient is finite,
    the formula's to half a step of the type, one of it and one of the products (see silu_terms)."""
    dev, tm = env
    N, H, I = 3, 64, 64
    d = DT[dt]
    x = torch.zeros(N, H, dtype=d)
    x[:, 0] = 1.0
    Wg, Wu = torch.zeros(I, H, dtype=d), torch.zeros(I, H, dtype=d)
    Wg[:, 0], Wu[:, 0] = -59.0, 1.07 * 2.0 ** 122
    Wd = torch.ones(H, I, dtype=d)
    L = [t.to(dev).requires_grad_() for t in (x, Wg, Wu, Wd)]
    y = tm.swiglu_ffn(*L, keep_activations="act8")
    assert bool(y.isfinite().all())
    y.backward(torch.ones_like(y))
    torch.cuda.synchronize()
    (h, tol), = R.silu_terms(torch.tensor([-60.0], dtype=torch.float64),
                             torch.tensor([1.125 * 2.0 ** 122], dtype=torch.float64))
    want = torch.full((H, I), float(N * h), dtype=torch.float64)
    # h^T is rounded to the type, then three of them are added and rounded once more
    R.check("dWd", L[3].grad, want, N * tol + (2 * R.half_step(d) + 4 * R.U32) * want.abs())


def test_keep8_no_tokens(env):
    dev, tm = env
    H, I, E = 64, 64, 4
    leaf = lambda *s: torch.randn(*s, device=dev).requires_grad_()
    x = torch.empty(0, H, device=dev).requires_grad_()
    L = [x, leaf(I, H), leaf(I, H), leaf(H, I)]
    tm.swiglu_ffn(*L, keep_activations="act8").sum().backward()
    M = [x, leaf(E, H), leaf(E, I, H), leaf(E, I, H), leaf(E, H, I)]
    y, aux = tm.moe_ffn(*M, 2, 0.01, keep_activations="act8")[:2]
    (y.sum() + aux.sum()).backward()
    torch.cuda.synchronize()
    assert all(not t.grad.any() for t in L + M)


def test_keep8_holds_less(env):
    """What a training forward holds until the backward."""
    dev, tm = env
    N, H, I = 512, 256, 704
    L = [rnd(i, *s, dt=torch.bfloat16).to(dev).requires_grad_()
         for i, s in enumerate(((N, H), (I, H), (I, H), (H, I)))]
    held = {}
    for mode in (True, "act8", False):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y = tm.swiglu_ffn(*L, keep_activations=mode)
        held[mode] = torch.cuda.memory_allocated() - before
        del y
    assert held["act8"] <= held[False] + tm.ffn_keep8_bytes(N, H, I, torch.bfloat16) + 4096
    assert held["act8"] * 4 < held[True]


@pytest.mark.parametrize("kind", ["dense", "moe"])
def test_keep8_released_by_the_backward(env, kind):
    """The kept bytes are a saved tensor of the graph: gone after its backward while the output
    still holds it, there again for a second pass where the graph is retained, seen by hooks."""
    dev, tm = env
    announce(f"kept bytes after the backward, {kind}")
    N, H, I, E, k = 512, 256, 704, 4, 2
    d = torch.bfloat16
    if kind == "dense":
        shapes, kept = ((N, H), (I, H), (I, H), (H, I)), tm.ffn_keep8_bytes(N, H, I, d)
        run = lambda L: tm.swiglu_ffn(*L, keep_activations="act8")
    else:
        shapes = ((N, H), (E, H), (E, I, H), (E, I, H), (E, H, I))
        kept = tm.moe_keep8_bytes(N, H, I, E, k, d)
        run = lambda L: tm.moe_ffn(*L, k, 0.0, keep_activations="act8")[0]
    L = [rnd(i, *s, dt=torch.float32 if s == (E, H) else d, scale=0.1).to(dev).requires_grad_()
         for i, s in enumerate(shapes)]
    dy = rnd(9, N, H, dt=d).to(dev)
    for t in L:
        t.grad = torch.zeros_like(t)  # so that the gradients take no new memory
    seen = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(t.numel()) or t, lambda t: t):
        y = run(L)
    assert kept in seen
    y = run(L)
    y.backward(dy, retain_graph=True)
    first = [t.grad.clone() for t in L]
    for t in L:
        t.grad.zero_()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y.backward(dy)
    torch.cuda.synchronize()
    assert before - torch.cuda.memory_allocated() >= kept
    assert all(eq(t.grad, g) for t, g in zip(L, first))
    with pytest.raises(RuntimeError):
        y.backward(dy)


def test_keep8_captured(env):
    """The training step with kept bytes in a graph, replayed over new inputs."""
    dev, tm = env
    N, H, I = 130, 128, 192
    d = torch.bfloat16
    T = [rnd(i, *s, dt=d, scale=sc).to(dev) for i, (s, sc) in enumerate(
        (((N, H), 1.0), ((I, H), 0.1), ((I, H), 0.1), ((H, I), 0.1), ((N, H), 1.0)))]
    saved = torch.empty(tm.ffn_bwd_workspace_bytes(N, H, I, d), dtype=torch.uint8, device=dev)

    def step():
        y = tm.ffn_swiglu_fwd(*T[:4], saved=saved)
        kept = tm.ffn_swiglu_keep8(saved, N, H, I, d)
        tm.ffn_swiglu_restore8(kept, N, H, I, d, workspace=saved)
        b = tm.ffn_swiglu_bwd(*T[:4], T[4], workspace=saved, from_saved=True)
        return [y, kept, b.dx, b.dWg, b.dWu, b.dWd]

    x2 = rnd(9, N, H, dt=d).to(dev)
    x1 = T[0].clone()
    want = {}
    for name, x in (("1", x1), ("2", x2)):
        T[0].copy_(x)
        want[name] = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for r in range(4):
        name, x = ("1", x1) if r % 2 == 0 else ("2", x2)
        T[0].copy_(x)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        # the kept buffer's alignment gaps are not written
        assert all(eq(a, b) for a, b in zip(outs[:1] + outs[2:], want[name][:1] + want[name][2:]))
        torch.randn(1 << 16, device=dev).sum().item()
