"""The block operators' measured cases: dispatch / combine of tokens by expert, the norms around a
block with its gate and residual scale, and activations kept in 8 bits.

``run`` computes a case in elementary torch operations (32 bits, rounded once at the end) or, where
``own`` is set, with the library's entry points; ``exact`` gives the definitions' values in 64 bits.
All inputs come from a seed.
"""
import math

import torch

own = False

GROUP = 32  # elements that share one 8-bit scale
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# The most one pass may move: the largest listed case.
_MOST_BYTES = 1.1e9


def listed():
    return [
        # one generated token: the norm before the FFN, all latency
        {"name": "prenorm_token", "op": "prenorm", "dir": "fwd", "N": 1, "H": 2048, "dtype": "bf16"},
        # a short fp32 training batch: the norm's gradient joined with the residual stream's
        {"name": "prenorm_bwd_fp32", "op": "prenorm", "dir": "bwd", "N": 100, "H": 768, "dtype": "fp32"},
        # prefill / training batch between two blocks: norm after, channel gate, residual, next norm
        {"name": "postnorm_train", "op": "postnorm", "dir": "fwd", "N": 16384, "H": 2048,
         "dtype": "bf16", "norm": True, "gate": "channel", "next": True, "scale": 1.0},
        # its backward pass: both norms' gradients, the gate's and the weights'
        {"name": "postnorm_train_bwd", "op": "postnorm", "dir": "bwd", "N": 16384, "H": 2048,
         "dtype": "bf16", "norm": True, "gate": "channel", "next": True, "scale": 1.0},
        # decode batch of 32 tokens, 16 experts: rows for the experts, all latency
        {"name": "dispatch_decode", "op": "dispatch", "dir": "fwd", "N": 32, "H": 2048, "E": 16,
         "k": 2, "dtype": "bf16", "cap": 0.0, "pad": 0.0, "skew": 0.5},
        # prefill with about 10x between the fullest and the emptiest expert
        {"name": "dispatch_prefill", "op": "dispatch", "dir": "fwd", "N": 16384, "H": 768, "E": 8,
         "k": 2, "dtype": "bf16", "cap": 0.0, "pad": 0.0, "skew": 0.7},
        # fine-grained experts in fp32, a ragged batch under a capacity: the gradient of the rows
        {"name": "dispatch_bwd_fp32", "op": "dispatch", "dir": "bwd", "N": 4099, "H": 768, "E": 64,
         "k": 6, "dtype": "fp32", "cap": 1.25, "pad": 0.03, "skew": 0.5},
        # decode: the experts' rows back to 32 tokens with the residual stream
        {"name": "combine_decode", "op": "combine", "dir": "fwd", "N": 32, "H": 2048, "E": 16, "k": 2,
         "dtype": "bf16", "cap": 0.0, "pad": 0.0, "skew": 0.5, "residual": True},
        # training batch: gradients of the experts' rows and of the weights
        {"name": "combine_train_bwd", "op": "combine", "dir": "bwd", "N": 16384, "H": 2048, "E": 16,
         "k": 2, "dtype": "bf16", "cap": 0.0, "pad": 0.0, "skew": 0.5, "residual": False},
        # dense training step at full size: SwiGLU on a fused projection's two halves, kept in 8 bits
        {"name": "swiglu8_train", "op": "swiglu8", "dir": "fwd", "N": 16384, "C": 6464,
         "dtype": "bf16"},
        # its backward pass from the kept bytes, with h again for the down projection's gradient
        {"name": "swiglu8_train_bwd", "op": "swiglu8", "dir": "bwd", "N": 16384, "C": 6464,
         "dtype": "bf16"},
        # a small fp32 activation put away in 8 bits and restored
        {"name": "act8_fp32", "op": "act8", "dir": "both", "N": 100, "C": 2432, "dtype": "fp32"},
    ]


def _log_size(rng, lo, hi, multiple=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(multiple, int(round(v / multiple)) * multiple)


def draw(rng):
    """A case from the listed ones' ranges: 1 to 32768 rows, 64 to 8192 channels, up to 256 experts."""
    while True:
        op = rng.choice(["prenorm", "postnorm", "dispatch", "combine", "swiglu8", "act8"])
        c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "N": _log_size(rng, 1, 32768),
             "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        if op in ("prenorm", "postnorm", "dispatch", "combine"):
            c["H"] = _log_size(rng, 64, 8192, 8)
        if op == "postnorm":
            c["norm"] = rng.random() < 0.75
            c["gate"] = rng.choice(["none", "channel", "token", "rows"])
            c["next"] = rng.random() < 0.6
            c["scale"] = rng.choice([1.0, 1.0, 0.5, 1.75])
            if c["gate"] == "rows":  # one gate row per sequence of the batch
                c["groups"] = rng.choice([2, 3, 4, 8])
                c["N"] = max(1, c["N"] // c["groups"]) * c["groups"]
        if op in ("dispatch", "combine"):
            c["E"] = _log_size(rng, 1, 256)
            c["k"] = min(c["E"], rng.choice([1, 1, 2, 2, 4, 6, 8]))
            c["cap"] = rng.choice([0.0, 0.0, 1.0, 1.5])
            c["pad"] = rng.choice([0.0, 0.0, 0.1])
            c["skew"] = rng.uniform(0.0, 1.5)
            if op == "combine":
                c["residual"] = rng.random() < 0.5
        if op in ("swiglu8", "act8"):
            c["C"] = _log_size(rng, 64, 16384, 8)
        if op == "act8":
            c["dir"] = "both"
        if work(c)["bytes"] <= _MOST_BYTES:
            return c


def work(case):
    """Bytes with every input read once and every output written once, and the arithmetic."""
    es = 2 if case["dtype"] == "bf16" else 4
    op, fwd = case["op"], case["dir"] == "fwd"
    N = case["N"]
    if op in ("swiglu8", "act8"):
        n = N * case["C"]
        q = n + N * -(-case["C"] // GROUP)  # kept bytes with their scales
        if op == "act8":
            return {"bytes": 2 * (n * es + q), "flops": 4 * n}
        return {"bytes": 3 * n * es + 2 * q if fwd else 4 * n * es + 2 * q, "flops": 12 * n}
    H = case["H"]
    row = N * H * es
    if op == "prenorm":
        return {"bytes": 2 * row + H * es + 4 * N if fwd else 4 * row + 2 * H * es + 4 * N,
                "flops": (4 if fwd else 8) * N * H}
    if op == "postnorm":
        gate = {"none": 0, "channel": H, "token": N, "rows": case.get("groups", 1) * H}[case["gate"]]
        vec = (H * (case["norm"] + case["next"]) + gate) * es + 4 * N * (case["norm"] + case["next"])
        if fwd:
            return {"bytes": (3 + case["next"]) * row + vec, "flops": 10 * N * H}
        return {"bytes": (4 + 2 * case["next"]) * row + 2 * vec, "flops": 20 * N * H}
    rows, n = case["k"] * row, N * case["k"]
    if op == "dispatch":
        return {"bytes": row + rows + 12 * n + 4 * case["E"] if fwd else row + rows + 4 * n,
                "flops": 0 if fwd else n * H}
    if fwd:
        return {"bytes": rows + row * (2 if case["residual"] else 1) + 8 * n, "flops": 2 * n * H}
    return {"bytes": row + 2 * rows + 12 * n, "flops": 3 * n * H}


# ---------------------------------------------------------------- inputs
def _activations(g, N, H, dt, spread=1.0):
    """A residual stream: unit-scale channels, about one in 64 of them some ten times larger."""
    x = torch.randn(N, H, generator=g, device="cuda")
    big = torch.rand(H, generator=g, device="cuda") < 1 / 64
    return (x * spread * torch.where(big, 10.0, 1.0)).to(dt)


def _gradient(g, N, H, dt):
    return (torch.randn(N, H, generator=g, device="cuda") * 0.02).to(dt)


def _weight(g, H, dt):
    return (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dt)


def _routing(g, case):
    """Top-k choices and weights of a softmax router with per-expert offsets; padding tokens' entries are -1."""
    N, E, k = case["N"], case["E"], case["k"]
    logits = torch.randn(N, E, generator=g, device="cuda")
    logits = logits + case["skew"] * torch.randn(E, generator=g, device="cuda")
    p, idx = torch.topk(torch.softmax(logits, -1), k, dim=-1)
    idx = idx.to(torch.int32)
    pad = torch.rand(N, generator=g, device="cuda") < case["pad"]
    idx = torch.where(pad[:, None], torch.full_like(idx, -1), idx)
    return idx.contiguous(), (p / p.sum(-1, keepdim=True)).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    dt, N, fwd = DTYPES[case["dtype"]], case["N"], case["dir"] == "fwd"
    s = {"case": case, "dt": dt}
    op = case["op"]
    if op == "act8":
        s["x"] = _activations(g, N, case["C"], dt)
        return s
    if op == "swiglu8":
        C = case["C"]
        gu = _activations(g, N, 2 * C, dt)  # one projection's output, [g | u]
        s["g"], s["u"] = gu[:, :C], gu[:, C:]
        if not fwd:
            s["gq"], s["gs"] = _to8(s.pop("g").float())
            s["uq"], s["us"] = _to8(s.pop("u").float())
            s["dh"] = _gradient(g, N, C, dt)
        return s
    H = case["H"]
    if op == "prenorm":
        s["x"], s["w"] = _activations(g, N, H, dt, 2.0), _weight(g, H, dt)
        if not fwd:
            s["rstd"] = _rstd(s["x"].float())
            s["dn"], s["dres"] = _gradient(g, N, H, dt), _gradient(g, N, H, dt)
        return s
    if op == "postnorm":
        s["y"], s["res"] = _activations(g, N, H, dt, 0.5), _activations(g, N, H, dt, 2.0)
        s["w"] = _weight(g, H, dt) if case["norm"] else None
        s["next_w"] = _weight(g, H, dt) if case["next"] else None
        shape = {"none": None, "channel": (H,), "token": (N, 1),
                 "rows": (case.get("groups", 1), H)}[case["gate"]]
        s["gate"] = None if shape is None else torch.rand(shape, generator=g, device="cuda").to(dt)
        if not fwd:
            f = _postnorm(s)
            s["out"], s["rstd"], s["next_rstd"] = f["out"], f["rstd"], f["next_rstd"]
            s["dout"] = _gradient(g, N, H, dt)
            s["dn"] = _gradient(g, N, H, dt) if case["next"] else None
        return s
    s["idx"], s["alpha"] = _routing(g, case)
    if op == "dispatch" and fwd:
        s["x"] = _activations(g, N, H, dt)
        return s
    s["entry_row"] = _rows(s["idx"], case["E"], _capacity(case))[2]
    rows = N * case["k"]
    if op == "dispatch":
        s["dxs"] = _gradient(g, rows, H, dt)
        return s
    s["ys"] = _activations(g, rows, H, dt, 0.5)
    if fwd:
        s["res"] = _activations(g, N, H, dt, 2.0) if case["residual"] else None
    else:
        s["dy"] = _gradient(g, N, H, dt)
    return s


# ---------------------------------------------------------------- plain forms
def _capacity(case):
    """Entries an expert keeps, or None."""
    if case["cap"] <= 0:
        return None
    return math.ceil(case["cap"] * case["N"] * case["k"] / case["E"])


def _rows(idx, E, cap):
    """offsets [E + 1], row -> entry (-1 past the kept rows), entry -> row (-1 - row where not kept)."""
    flat = idx.reshape(-1).long()
    n, dev = flat.numel(), flat.device
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    counts = (key[:, None] == torch.arange(E + 1, device=dev)).sum(0)
    first = counts.cumsum(0) - counts
    order = torch.argsort(key, stable=True)
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(n, device=dev) - first[key[order]]
    most = counts if cap is None else counts.clamp(max=cap)
    most = torch.where(torch.arange(E + 1, device=dev) < E, most, torch.zeros_like(most))
    off = most.cumsum(0) - most
    left = counts - most
    tail = most.sum() + left.cumsum(0) - left
    kept = rank < most[key]
    row = torch.where(kept, off[key] + rank, tail[key] + rank - most[key])
    row_entry = torch.empty_like(flat)
    row_entry[row] = torch.where(kept, torch.arange(n, device=dev), torch.full_like(flat, -1))
    entry_row = torch.where(kept, row, -1 - row).reshape(idx.shape)
    return off.to(torch.int32), row_entry.to(torch.int32), entry_row.to(torch.int32)


def _rstd(x):
    return torch.rsqrt((x * x).mean(-1) + EPS)


def _gate(s):
    """The gate as [N or 1, H or 1] in float32, 1 where there is none."""
    case, gate = s["case"], s["gate"]
    if gate is None:
        return torch.ones(1, 1, device="cuda")
    gate = gate.float()
    if case["gate"] == "rows":
        return gate.repeat_interleave(case["N"] // case["groups"], 0)
    return gate if case["gate"] == "token" else gate[None]


def _postnorm(s):
    y, res = s["y"].float(), s["res"].float()
    rstd = next_rstd = n = None
    b = y
    if s["w"] is not None:
        rstd = _rstd(y)
        b = y * rstd[:, None] * s["w"].float()
    r = s["case"]["scale"] * res + _gate(s) * b
    if s["next_w"] is not None:
        next_rstd = _rstd(r)
        n = (r * next_rstd[:, None] * s["next_w"].float()).to(s["dt"])
    return {"out": r.to(s["dt"]), "rstd": rstd, "n": n, "next_rstd": next_rstd}


def _postnorm_bwd(s):
    case, dt = s["case"], s["dt"]
    y, dr, gate = s["y"].float(), s["dout"].float(), _gate(s)
    dnext_w = dw = dgate = None
    if s["next_w"] is not None:
        rh, dn = s["out"].float() * s["next_rstd"][:, None], s["dn"].float()
        a = dn * s["next_w"].float()
        dr = dr + s["next_rstd"][:, None] * (a - rh * (a * rh).mean(-1, keepdim=True))
        dnext_w = (dn * rh).sum(0).to(dt)
    yh, b, wg = y, dr * gate, dr * y
    if s["w"] is not None:
        yh = y * s["rstd"][:, None]
        dw = (dr * gate * yh).sum(0).to(dt)
        b, wg = b * s["w"].float(), dr * yh * s["w"].float()
        dy = s["rstd"][:, None] * (b - yh * (b * yh).mean(-1, keepdim=True))
    else:
        dy = b
    if case["gate"] == "token":
        dgate = wg.sum(-1, keepdim=True).to(dt)
    elif case["gate"] == "channel":
        dgate = wg.sum(0).to(dt)
    elif case["gate"] == "rows":
        dgate = wg.reshape(case["groups"], -1, case["H"]).sum(1).to(dt)
    return {"dy": dy.to(dt), "dres": (case["scale"] * dr).to(dt), "dw": dw, "dgate": dgate,
            "dnext_w": dnext_w}


def _to8(x):
    """e4m3 values and their scale bytes: groups of 32 channels, the smallest power of two that brings
    the group's largest finite magnitude to 448 or less; elements that are not finite become NaN."""
    N, C = x.shape
    G = -(-C // GROUP)
    fine = torch.isfinite(x)
    mag = torch.nn.functional.pad(torch.where(fine, x.abs(), torch.zeros_like(x)), (0, G * GROUP - C))
    bits = mag.reshape(N, G, GROUP).amax(-1).view(torch.int32)
    e = ((bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=-127)
    scaled = torch.ldexp(x, -e.repeat_interleave(GROUP, 1)[:, :C])
    q = torch.where(fine, scaled, torch.full_like(x, math.nan)).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _from8(q, scale):
    e = scale.to(torch.int32) - 127
    return torch.ldexp(q.float(), e.repeat_interleave(GROUP, 1)[:, :q.shape[1]])


def _kept(entry_row):
    """(row, kept as 0 / 1) of every entry, rows of entries not kept included."""
    row = entry_row.long()
    return torch.where(row < 0, -1 - row, row), (row >= 0).float()


def _plain(s):
    case, dt = s["case"], s["dt"]
    op, fwd = case["op"], case["dir"] == "fwd"
    if op == "act8":
        q, scale = _to8(s["x"].float())
        return {"q": q, "scale": scale, "x": _from8(q, scale).to(dt)}
    if op == "swiglu8" and fwd:
        g, u = s["g"].float(), s["u"].float()
        gq, gs = _to8(g)
        uq, us = _to8(u)
        return {"h": (g * torch.sigmoid(g) * u).to(dt), "gq": gq, "gs": gs, "uq": uq, "us": us}
    if op == "swiglu8":
        g, u, dh = _from8(s["gq"], s["gs"]), _from8(s["uq"], s["us"]), s["dh"].float()
        sig = torch.sigmoid(g)
        return {"dg": (dh * u * sig * (1 + g * (1 - sig))).to(dt), "du": (dh * g * sig).to(dt),
                "h": (g * sig * u).to(dt)}
    if op == "prenorm":
        x, w = s["x"].float(), s["w"].float()
        if fwd:
            rstd = _rstd(x)
            return {"n": (x * rstd[:, None] * w).to(dt), "rstd": rstd}
        rstd, dn = s["rstd"][:, None], s["dn"].float()
        xh, a = x * rstd, dn * w
        dx = s["dres"].float() + rstd * (a - xh * (a * xh).mean(-1, keepdim=True))
        return {"dx": dx.to(dt), "dw": (dn * xh).sum(0).to(dt)}
    if op == "postnorm":
        return _postnorm(s) if fwd else _postnorm_bwd(s)
    N, k, H = case["N"], case["k"], case["H"]
    if op == "dispatch" and fwd:
        off, row_entry, entry_row = _rows(s["idx"], case["E"], _capacity(case))
        xs = s["x"][(row_entry.long() // k).clamp(min=0)]
        xs = torch.where((row_entry >= 0)[:, None], xs, torch.zeros_like(xs))
        return {"xs": xs, "offsets": off, "row_entry": row_entry, "entry_row": entry_row}
    row, kept = _kept(s["entry_row"])
    if op == "dispatch":
        return {"dx": (s["dxs"].float()[row.reshape(-1)].reshape(N, k, H) * kept[..., None]).sum(1).to(dt)}
    ys = s["ys"].float()[row.reshape(-1)].reshape(N, k, H)
    wt = s["alpha"] * kept
    if fwd:
        y = (ys * wt[..., None]).sum(1)
        return {"y": (y if s["res"] is None else y + s["res"].float()).to(dt)}
    dy = s["dy"].float()
    dys = torch.empty(N * k, H, dtype=dt, device="cuda")
    dys[row.reshape(-1)] = (dy[:, None] * wt[..., None]).reshape(N * k, H).to(dt)
    return {"dys": dys, "dalpha": (dy[:, None] * ys).sum(-1) * kept}


# ---------------------------------------------------------------- the library's operators
def _library(s):
    import top_moe_layer_amd as tm

    case = s["case"]
    op, fwd = case["op"], case["dir"] == "fwd"
    if op == "act8":
        a = tm.act8_pack(s["x"])
        return {"q": a.q, "scale": a.scale, "x": tm.act8_unpack(a.q, a.scale, dtype=s["dt"])}
    if op == "swiglu8" and fwd:
        o = tm.swiglu_act8_fwd(s["g"], s["u"])
        return {"h": o.h, "gq": o.g8.q, "gs": o.g8.scale, "uq": o.u8.q, "us": o.u8.scale}
    if op == "swiglu8":
        o = tm.swiglu_act8_bwd(s["dh"], tm.Act8(s["gq"], s["gs"]), tm.Act8(s["uq"], s["us"]))
        return {"dg": o.dg, "du": o.du, "h": o.h}
    if op == "prenorm" and fwd:
        o = tm.block_prenorm_fwd(s["x"], s["w"], eps=EPS)
        return {"n": o.n, "rstd": o.rstd}
    if op == "prenorm":
        o = tm.block_prenorm_bwd(s["dn"], s["x"], s["w"], s["rstd"], dresidual=s["dres"])
        return {"dx": o.dx, "dw": o.dw}
    if op == "postnorm" and fwd:
        o = tm.block_postnorm_fwd(s["y"], s["res"], s["w"], gate=s["gate"], next_w=s["next_w"],
                                  residual_scale=case["scale"], eps=EPS)
        return {"out": o.out, "rstd": o.rstd, "n": o.n, "next_rstd": o.next_rstd}
    if op == "postnorm":
        o = tm.block_postnorm_bwd(s["dout"], s["y"], s["w"], rstd=s["rstd"], gate=s["gate"],
                                  dn=s["dn"], out=s["out"], next_w=s["next_w"],
                                  next_rstd=s["next_rstd"], residual_scale=case["scale"])
        return {"dy": o.dy, "dres": o.dresidual, "dw": o.dw, "dgate": o.dgate, "dnext_w": o.dnext_w}
    if op == "dispatch" and fwd:
        o = tm.moe_dispatch_fwd(s["x"], s["idx"], case["E"], capacity_factor=case["cap"])
        return {"xs": o.xs, "offsets": o.expert_offsets, "row_entry": o.row_entry,
                "entry_row": o.entry_row}
    if op == "dispatch":
        return {"dx": tm.moe_dispatch_bwd(s["dxs"], s["entry_row"])}
    if fwd:
        return {"y": tm.moe_combine_fwd(s["ys"], s["entry_row"], s["alpha"], residual=s["res"])}
    o = tm.moe_combine_bwd(s["dy"], s["ys"], s["entry_row"], s["alpha"])
    return {"dys": o.dys, "dalpha": o.dalpha}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits
def _exact_8(x):
    """(e4m3 values, exponents) of [N, C] in 64 bits, by the grid's spacing."""
    N, C = x.shape
    x = x.double()
    fine = torch.isfinite(x)
    ex = torch.empty(N, C, device=x.device, dtype=torch.float64)
    for c in range(0, C, GROUP):  # the smallest 2^e with largest <= 448 * 2^e
        a = torch.where(fine[:, c:c + GROUP], x[:, c:c + GROUP].abs(), 0.0).amax(1, keepdim=True)
        ex[:, c:c + GROUP] = torch.ceil(torch.log2(a / 448.0)).clamp(min=-127)
    v = x * torch.exp2(-ex)
    over = v.abs() > 448.0  # log2 of a value next to a power of two may be off in its last bit
    ex = torch.where(over, ex + 1, ex)
    v = torch.where(over, v / 2, v)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(v / step) * step
    return torch.where(fine, q, math.nan), ex


def _exact_silu(g):
    return g / (1 + torch.exp(-g))


def exact(case, seed):
    s = prepare(case, seed)
    op, fwd, N = case["op"], case["dir"] == "fwd", case["N"]
    if op == "act8":
        q, ex = _exact_8(s["x"])
        return {"q": q, "scale": None, "x": q * torch.exp2(ex)}
    if op == "swiglu8" and fwd:
        g, u = s["g"].double(), s["u"].double()
        return {"h": _exact_silu(g) * u, "gq": _exact_8(g)[0], "gs": None, "uq": _exact_8(u)[0],
                "us": None}
    if op == "swiglu8":
        C = case["C"]
        at = torch.arange(C, device="cuda") // GROUP
        g = s["gq"].double() * torch.exp2(s["gs"].double() - 127)[:, at]
        u = s["uq"].double() * torch.exp2(s["us"].double() - 127)[:, at]
        dh, ex = s["dh"].double(), torch.exp(-g)
        return {"dg": dh * u * (1 / (1 + ex) + g * ex / (1 + ex) ** 2), "du": dh * _exact_silu(g),
                "h": _exact_silu(g) * u}
    if op == "prenorm":
        x, w = s["x"].double(), s["w"].double()
        if fwd:
            rms = (x.square().sum(1) / case["H"] + EPS).sqrt()
            return {"n": x / rms[:, None] * w, "rstd": 1 / rms}
        r, dn = s["rstd"].double()[:, None], s["dn"].double()
        inner = (dn * w * x).sum(1, keepdim=True)
        return {"dx": s["dres"].double() + r * dn * w - x * r ** 3 * inner / case["H"],
                "dw": (dn * x * r).sum(0)}
    if op == "postnorm":
        return _exact_postnorm(s, fwd)
    k, H, E = case["k"], case["H"], case["E"]
    if op == "dispatch" and fwd:
        cap, flat = _capacity(case), s["idx"].reshape(-1)
        lists = [torch.nonzero(flat == e).flatten()[:cap] for e in range(E)]
        order = torch.cat(lists)
        xs = torch.zeros(N * k, H, dtype=torch.float64, device="cuda")
        xs[:order.numel()] = s["x"].double()[order // k]
        return {"xs": xs, "offsets": None, "row_entry": None, "entry_row": None}
    er = s["entry_row"].long()
    if op == "dispatch":
        dx = torch.zeros(N, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(er[:, j] >= 0).flatten()
            dx[t] += s["dxs"].double()[er[t, j]]
        return {"dx": dx}
    alpha, ys = s["alpha"].double(), s["ys"]
    if fwd:
        y = torch.zeros(N, H, dtype=torch.float64, device="cuda") if s["res"] is None else s["res"].double()
        for j in range(k):
            t = torch.nonzero(er[:, j] >= 0).flatten()
            y[t] += alpha[t, j, None] * ys[er[t, j]].double()
        return {"y": y}
    dy = s["dy"].double()
    dys = torch.zeros(N * k, H, dtype=torch.float64, device="cuda")
    dalpha = torch.zeros(N, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(er[:, j] >= 0).flatten()
        dys[er[t, j]] = alpha[t, j, None] * dy[t]
        dalpha[t, j] = (dy[t] * ys[er[t, j]].double()).sum(1)
    return {"dys": dys, "dalpha": dalpha}


def _exact_postnorm(s, fwd):
    """By the chain rule in 64 bits, each token's gate spread to a row of its own."""
    case = s["case"]
    N, H = case["N"], case["H"]
    y = s["y"].double()
    if s["gate"] is None:
        gate = torch.ones(N, H, dtype=torch.float64, device="cuda")
    else:
        gate = s["gate"].double()
        if case["gate"] == "rows":
            gate = gate[torch.arange(N, device="cuda") // (N // case["groups"])]
        gate = gate.expand(N, H)
    w = s["w"].double() if case["norm"] else torch.ones(H, dtype=torch.float64, device="cuda")
    if fwd:
        rms = (y.square().sum(1) / H + EPS).sqrt() if case["norm"] else torch.ones(N, device="cuda")
        r = case["scale"] * s["res"].double() + gate * (y / rms[:, None]) * w
        o = {"out": r, "rstd": 1 / rms if case["norm"] else None, "n": None, "next_rstd": None}
        if case["next"]:
            rms = (r.square().sum(1) / H + EPS).sqrt()
            o["n"], o["next_rstd"] = r / rms[:, None] * s["next_w"].double(), 1 / rms
        return o
    dr, dnext_w = s["dout"].double(), None
    if case["next"]:
        r, k, dn, v = s["out"].double(), s["next_rstd"].double()[:, None], s["dn"].double(), s["next_w"].double()
        dr = dr + k * dn * v - r * k ** 3 * (dn * v * r).sum(1, keepdim=True) / H
        dnext_w = (dn * r * k).sum(0)
    c = s["rstd"].double()[:, None] if case["norm"] else torch.ones(N, 1, dtype=torch.float64, device="cuda")
    b = dr * gate * w
    dy = c * b
    if case["norm"]:
        dy = dy - y * c ** 3 * (b * y).sum(1, keepdim=True) / H
    each = dr * w * y * c  # the gate's gradient, channel by channel
    dgate = {"none": lambda: None, "channel": lambda: each.sum(0), "token": lambda: each.sum(1, keepdim=True),
             "rows": lambda: each.view(case.get("groups", 1), -1, H).sum(1)}[case["gate"]]()
    return {"dy": dy, "dres": case["scale"] * dr, "dw": (dr * gate * y * c).sum(0) if case["norm"] else None,
            "dgate": dgate, "dnext_w": dnext_w}
