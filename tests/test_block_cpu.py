"""Refusals of the block operators that need no GPU: the C ABI validates on the
host before anything is launched, the torch front end before that."""
import math

import pytest
import torch

import top_moe_layer_amd as tm
from top_moe_layer_amd import _binding as B

FAKE = 1 << 20  # 256-byte aligned, never dereferenced: validation fails first
BF16 = B.DTYPE_BF16
NAN, INF = float("nan"), float("inf")


def call(name, base, **over):
    a = dict(base)
    assert set(over) <= set(a), set(over) - set(a)
    a.update(over)
    return getattr(B.lib(), name)(*a.values(), None, None)


DISPATCH = dict(x=FAKE, idx=FAKE, N=32768, H=64, E=4, k=2, cf=0.0, dtype=BF16, xs=FAKE, off=FAKE,
                row_entry=FAKE, entry_row=FAKE, ws=FAKE, ws_bytes=0)
DISPATCH_BWD = dict(dxs=FAKE, entry_row=FAKE, N=8, H=64, k=2, dtype=BF16, dx=None)
COMBINE = dict(ys=FAKE, entry_row=FAKE, alpha=FAKE, residual=None, N=8, H=64, k=2, dtype=BF16,
               y=None)
COMBINE_BWD = dict(dy=FAKE, ys=FAKE, entry_row=FAKE, alpha=FAKE, N=8, H=64, k=2, dtype=BF16,
                   dys=FAKE, dalpha=None)
PRE = dict(x=FAKE, w=FAKE, N=8, H=64, eps=1e-5, dtype=BF16, n=FAKE, rstd=None)
PRE_BWD = dict(dn=FAKE, x=FAKE, w=FAKE, rstd=FAKE, dres=None, N=8, H=64, dtype=BF16, dx=FAKE,
               dw=FAKE, ws=FAKE, ws_bytes=0)
POST = dict(y=FAKE, residual=FAKE, w=FAKE, gate=FAKE, next_w=FAKE, N=8, H=64, mode=1, rows=2,
            scale=1.0, eps=1e-5, dtype=BF16, out=FAKE, rstd=FAKE, n=FAKE, next_rstd=None)
POST_BWD = dict(dout=FAKE, dn=FAKE, y=FAKE, out=FAKE, w=FAKE, gate=FAKE, next_w=FAKE, rstd=FAKE,
                next_rstd=FAKE, N=8, H=64, mode=1, rows=2, scale=1.0, dtype=BF16, dy=FAKE,
                dres=FAKE, dw=FAKE, dgate=FAKE, dnext_w=FAKE, ws=FAKE, ws_bytes=0)
PACK = dict(x=FAKE, ldx=64, R=8, C=64, dtype=BF16, q=FAKE, scale=None)
UNPACK = dict(q=FAKE, scale=None, R=8, C=64, dtype=BF16, x=FAKE, ldx=64)
SWIGLU = dict(g=FAKE, ldg=64, u=FAKE, ldu=64, R=8, C=64, dtype=BF16, h=FAKE, gq=FAKE, gs=FAKE,
              uq=FAKE, us=None)
SWIGLU_BWD = dict(gq=FAKE, gs=FAKE, uq=FAKE, us=FAKE, dh=FAKE, R=8, C=64, dtype=BF16, dg=FAKE,
                  lddg=64, du=None, lddu=64, h=None)
ALL = {"moe_dispatch_fwd": DISPATCH, "moe_dispatch_bwd": DISPATCH_BWD, "moe_combine_fwd": COMBINE,
       "moe_combine_bwd": COMBINE_BWD, "block_prenorm_fwd": PRE, "block_prenorm_bwd": PRE_BWD,
       "block_postnorm_fwd": POST, "block_postnorm_bwd": POST_BWD, "act8_pack": PACK,
       "act8_unpack": UNPACK, "swiglu_act8_fwd": SWIGLU, "swiglu_act8_bwd": SWIGLU_BWD}


@pytest.mark.parametrize("name", ALL)
def test_common_refusals(name):
    base = ALL[name]
    # each base call is complete but for one thing: a missing output or too small a workspace
    want = B.ERR_WORKSPACE_TOO_SMALL if "ws" in base else B.ERR_NULL_ARG
    assert call(name, base) == want
    assert call(name, base, dtype=2) == B.ERR_UNSUPPORTED_DTYPE
    assert call(name, base, dtype=-1) == B.ERR_UNSUPPORTED_DTYPE
    rows, cols = ("R", "C") if "R" in base else ("N", "H")
    for over in ({rows: -1}, {rows: 1 << 31}, {cols: 0}, {cols: -8}, {cols: 60}, {cols: 1 << 31}):
        assert call(name, base, **over) == B.ERR_BAD_SHAPE, over


@pytest.mark.parametrize("name", ["moe_dispatch_fwd", "moe_dispatch_bwd", "moe_combine_fwd",
                                  "moe_combine_bwd"])
def test_rows_refusals(name):
    base = ALL[name]
    for over in (dict(k=0), dict(k=257), dict(N=(1 << 30), k=2), dict(H=(1 << 20) + 8)):
        assert call(name, base, **over) == B.ERR_BAD_SHAPE, over
    if "E" in base:
        for over in (dict(E=0), dict(E=257), dict(k=5)):
            assert call(name, base, **over) == B.ERR_BAD_SHAPE, over
        for cf in (-1.0, NAN, INF):
            assert call(name, base, cf=cf) == B.ERR_BAD_ARG
        need = tm.moe_dispatch_workspace_bytes(32768, 4, 2)
        # few entries of long rows take three launches as well: 1024 * 3 * 2^15 * 2 bytes
        assert call(name, base, N=1024, H=1 << 15) == B.ERR_WORKSPACE_TOO_SMALL
        assert call(name, base, ws_bytes=64 * 4) == B.ERR_WORKSPACE_TOO_SMALL
        assert call(name, base, ws=None) == B.ERR_NULL_ARG
        for p, off in (("x", 8), ("xs", 8), ("idx", 2), ("off", 1), ("entry_row", 2), ("ws", 64)):
            assert call(name, base, ws_bytes=need, **{p: FAKE + off}) == B.ERR_BAD_ARG, p


def test_dispatch_workspace():
    assert tm.moe_dispatch_workspace_bytes(0, 1, 1) >= 1
    # 256 chunks of counts at most
    assert tm.moe_dispatch_workspace_bytes((1 << 31) - 1, 256, 1) <= 256 * 257 * 4 + 512
    for bad in ((-1, 4, 2), (8, 0, 1), (8, 257, 1), (8, 4, 5), (8, 4, 0), (1 << 30, 4, 2)):
        assert tm.moe_dispatch_workspace_bytes(*bad) == 0, bad


def test_norm_refusals():
    for eps in (0.0, -1e-6, NAN, INF):
        assert call("block_prenorm_fwd", PRE, rstd=FAKE, eps=eps) == B.ERR_BAD_ARG
        assert call("block_postnorm_fwd", POST, next_rstd=FAKE, eps=eps) == B.ERR_BAD_ARG
    for name in ("block_prenorm_fwd", "block_prenorm_bwd", "block_postnorm_fwd",
                 "block_postnorm_bwd"):
        assert call(name, ALL[name], H=16392) == B.ERR_BAD_SHAPE
    for name in ("block_postnorm_fwd", "block_postnorm_bwd"):
        b = ALL[name]
        assert call(name, b, mode=3) == B.ERR_BAD_ARG
        assert call(name, b, mode=-1) == B.ERR_BAD_ARG
        for rows in (3, 0, -2, 16):
            assert call(name, b, rows=rows) == B.ERR_BAD_SHAPE, rows
        assert call(name, b, gate=None) == B.ERR_NULL_ARG
        assert call(name, b, rstd=None) == B.ERR_NULL_ARG
    assert call("block_postnorm_fwd", POST, next_rstd=FAKE, scale=NAN) == B.ERR_BAD_ARG
    assert call("block_postnorm_bwd", POST_BWD, scale=INF) == B.ERR_BAD_ARG
    for over in (dict(dn=None), dict(out=None), dict(next_rstd=None), dict(dw=None),
                 dict(dgate=None), dict(dnext_w=None), dict(dout=None, next_w=None),
                 dict(ws=None)):
        assert call("block_postnorm_bwd", POST_BWD, **over) == B.ERR_NULL_ARG, over
    # the gradient of n alone needs no dout: the workspace check is the first to fail
    assert call("block_postnorm_bwd", POST_BWD, dout=None) == B.ERR_WORKSPACE_TOO_SMALL
    need = tm.block_norm_bwd_workspace_bytes(8, 64, 2)
    for p, off in (("dout", 8), ("dgate", 2), ("dw", 4), ("rstd", 2), ("ws", 128)):
        assert call("block_postnorm_bwd", POST_BWD, ws_bytes=need, **{p: FAKE + off}) == B.ERR_BAD_ARG, p
    assert tm.block_norm_bwd_workspace_bytes(8, 64, 3) == 0
    assert tm.block_norm_bwd_workspace_bytes(8, 60, 1) == 0
    assert tm.block_norm_bwd_workspace_bytes(0, 64, 5) > 0


def test_act8_refusals():
    assert call("act8_pack", PACK, ldx=56) == B.ERR_BAD_SHAPE
    assert call("act8_pack", PACK, ldx=68) == B.ERR_BAD_SHAPE
    assert call("act8_unpack", UNPACK, ldx=63) == B.ERR_BAD_SHAPE
    assert call("swiglu_act8_fwd", SWIGLU, ldu=60) == B.ERR_BAD_SHAPE
    assert call("swiglu_act8_bwd", SWIGLU_BWD, lddg=60) == B.ERR_BAD_SHAPE
    assert call("act8_pack", PACK, scale=FAKE, x=FAKE + 8) == B.ERR_BAD_ARG
    assert call("act8_pack", PACK, scale=FAKE, q=FAKE + 4) == B.ERR_BAD_ARG
    assert call("swiglu_act8_bwd", SWIGLU_BWD, du=FAKE, h=FAKE + 4) == B.ERR_BAD_ARG


def test_keep8_refusals():
    ffn = dict(src=FAKE, src_bytes=1 << 40, N=8, H=64, I=64, dtype=BF16, dst=FAKE, dst_bytes=0)
    moe = dict(src=FAKE, src_bytes=1 << 40, N=8, H=64, I=64, E=4, k=2, dtype=BF16, dst=FAKE,
               dst_bytes=0)
    for base, names in ((ffn, ("ffn_swiglu_keep8", "ffn_swiglu_restore8")),
                        (moe, ("moe_ffn_keep8", "moe_ffn_restore8"))):
        for name in names:
            assert call(name, base) == B.ERR_WORKSPACE_TOO_SMALL
            assert call(name, base, dst_bytes=1 << 40, src_bytes=255) == B.ERR_WORKSPACE_TOO_SMALL
            assert call(name, base, src=None) == B.ERR_NULL_ARG
            assert call(name, base, dst=None) == B.ERR_NULL_ARG
            assert call(name, base, dst_bytes=1 << 40, dst=FAKE + 128) == B.ERR_BAD_ARG
            assert call(name, base, dst_bytes=1 << 40, src=FAKE + 64) == B.ERR_BAD_ARG
            for over in (dict(I=96), dict(H=32), dict(N=-1)):
                assert call(name, base, **over) == B.ERR_BAD_SHAPE, over
            assert call(name, base, dtype=3) == B.ERR_UNSUPPORTED_DTYPE
    n = 16384 * 6464  # a sixteenth of a byte of scales for each two bytes
    assert 0 <= tm.ffn_keep8_bytes(16384, 2048, 6464, torch.bfloat16) - (2 * n + n // 16) <= 1024
    assert tm.moe_keep8_bytes(8, 64, 96, 4, 2, torch.bfloat16) == 0


def test_front_end_refusals():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: tm.block_prenorm_fwd(x, w), lambda: tm.moe_dispatch_fwd(x, idx, 4),
              lambda: tm.block_postnorm_fwd(x, x, w), lambda: tm.act8_pack(x),
              lambda: tm.moe_combine_fwd(x, idx, x), lambda: tm.swiglu_act8_fwd(x, x)):
        with pytest.raises(ValueError, match="no CPU path"):
            f()
    with pytest.raises(TypeError):
        tm.act8_pack([1.0])


@pytest.mark.parametrize("factor", [1.2, 0.6, 1.6, 1.1, 0.7, 1.25, 0.01, 1e-300, 5.0, 1e308])
def test_capacity_of_a_factor(factor):
    """Whole-number products of factors that 32 bits do not hold stay whole (1.2 as a float lies
    above 1.2)."""
    from top_moe_layer_amd import block

    for N, E, k in ((50, 10, 2), (500, 8, 2), (1000, 10, 1), (33, 5, 3), (1 << 20, 64, 8)):
        n = N * k
        c = factor * n / E
        assert (block._capacity(factor, N, E, k) or n) == (min(math.ceil(c), n) if c < n else n)
    assert block._capacity(1.2, 50, 10, 2) == 12
    assert block._capacity(0.0, 50, 10, 2) == 0
    for bad in (-1.0, NAN, INF):
        with pytest.raises(tm.TopmoeError):
            block._capacity(bad, 50, 10, 2)


def test_capacity_refusals():
    base = {("capacity" if n == "cf" else n): (0 if n == "cf" else v) for n, v in DISPATCH.items()}
    name = "moe_dispatch_fwd_capacity"
    assert call(name, base) == B.ERR_WORKSPACE_TOO_SMALL
    assert call(name, base, capacity=1 << 40) == B.ERR_WORKSPACE_TOO_SMALL
    assert call(name, base, capacity=-1) == B.ERR_BAD_ARG
    assert call(name, base, capacity=-(1 << 40)) == B.ERR_BAD_ARG
    assert call(name, base, dtype=2) == B.ERR_UNSUPPORTED_DTYPE
    assert call(name, base, E=0) == B.ERR_BAD_SHAPE
    assert call(name, base, xs=None) == B.ERR_NULL_ARG


def test_gate_shapes():
    """Rows of a gate belong to runs of consecutive tokens; what broadcasting would read otherwise
    is refused."""
    from top_moe_layer_amd import block

    H, dt, dev = 64, torch.float32, torch.device("cpu")

    def gate(shape, *lead):
        y = torch.zeros(*lead, H)
        return block._gate(torch.zeros(shape), y.shape, y.numel() // H, H, dt, dev)

    channel = lambda rows: (B.GATE_CHANNEL, rows)
    token = (B.GATE_TOKEN, 1)
    for shape, lead, want in [
            ((H,), (2, 4), channel(1)), ((2, H), (2, 4), channel(2)), ((4, H), (2, 4), channel(4)),
            ((1, H), (8,), channel(1)), ((2, 1, H), (2, 4), channel(2)), ((1, 1, H), (2, 4), channel(1)),
            ((4, 1, H), (2, 4), channel(4)), ((2, 4, H), (2, 4), channel(8)), ((1, 4, H), (1, 4), channel(4)),
            ((2, 1, H), (8,), channel(2)), ((2, 4, H), (8,), channel(8)), ((2, 3, 1, H), (2, 3, 4), channel(6)),
            ((2, 1, 1, H), (2, 3, 4), channel(2)), ((2, 1, 4, H), (2, 1, 4), channel(8)),
            ((1, H), (), channel(1)), ((1, 1, H), (), channel(1)), ((0, 1, H), (0, 4), channel(0)),
            ((8, 1), (8,), token), ((2, 4, 1), (2, 4), token), ((8, 1), (2, 4), token),
            ((1, 1), (1,), token), ((0, 1), (0,), token)]:
        assert gate(shape, *lead) == want, (shape, lead)
    for shape, lead in [((1, 4, H), (2, 4)), ((1, 4, H), (8,)), ((4, 2, H), (2, 4)),
                        ((2, 1, 4, H), (2, 3, 4)), ((1, 3, 1, H), (2, 3, 4)), ((3, H), (2, 4)),
                        ((4, 2, 1), (2, 4)), ((1, 4, 1), (2, 4)), ((4,), (4,))]:
        with pytest.raises(ValueError):
            gate(shape, *lead)


def test_too_few_stage_events():
    """Every entry point's stage count, and the refusal of events for fewer."""
    from top_moe_layer_amd import block, ops

    class Events(B.StageEvents):
        def __init__(self, stages):  # no events are made
            self.stages, self.n, self.arr = stages, 2 * stages, None

    assert set(block._STAGES) <= set(B.SIGNATURES)
    for name in ("block_prenorm_bwd", "moe_dispatch_fwd_capacity", "ffn_swiglu_restore8", "act8_pack"):
        stages = block._STAGES.get(name, 1)
        with pytest.raises(ValueError, match="stages"):
            block._call(name, torch.device("cuda", 0), Events(stages - 1))
    for stages in (B.FFN_STAGES, B.MOE_STAGES, B.FFN_BWD_STAGES, B.MOE_BWD_STAGES):
        with pytest.raises(ValueError, match="stages"):
            ops._events(Events(stages - 1), stages)
        assert ops._events(Events(stages), stages).value is None
    assert ops._events(None, 2) is None
