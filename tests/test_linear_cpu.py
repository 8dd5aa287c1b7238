"""Products by expert and 4-bit matrices without a GPU: refusals of the C ABI (validated on the host
before anything is launched) and of the torch front end, and the format's reference."""
import math

import pytest
import torch

import linear_ref as R
import top_moe_layer_amd as tm
from top_moe_layer_amd import _binding as B

FAKE = 1 << 20  # 256-byte aligned, never dereferenced: validation fails first
BF16 = B.DTYPE_BF16


def call(name, base, **over):
    a = dict(base)
    assert set(over) <= set(a), set(over) - set(a)
    a.update(over)
    return getattr(B.lib(), name)(*a.values(), None, None)


# each complete but for a missing output or too small a workspace
FWD = dict(x=FAKE, ldx=64, w=FAKE, off=FAKE, R=8, K=64, O=48, E=4, dtype=BF16, y=None, ldy=48)
BWD = dict(dy=FAKE, lddy=48, x=FAKE, ldx=64, w=FAKE, off=FAKE, R=8, K=64, O=48, E=4, dtype=BF16,
           dx=FAKE, lddx=64, dw=FAKE, ws=FAKE, ws_bytes=0)
PACK = dict(x=FAKE, ldx=64, R=8, C=64, dtype=BF16, q=FAKE, scale=None)
UNPACK = dict(q=FAKE, scale=None, R=8, C=64, dtype=BF16, x=FAKE, ldx=64)
MX = dict(x=FAKE, ldx=64, xs=None, rows=0, wq=FAKE, ws=FAKE, off=FAKE, R=8, K=64, O=48, E=4,
          dtype=BF16, y=None, ldy=48)
MX_BWD = dict(dy=FAKE, lddy=48, wq=FAKE, wscale=FAKE, off=FAKE, R=8, K=64, O=48, E=4, dtype=BF16,
              dx=FAKE, lddx=64, ws=FAKE, ws_bytes=0)
LINEAR = {"moe_linear_fwd": FWD, "moe_linear_bwd": BWD, "mx4_linear_fwd": MX,
          "mx4_linear_bwd": MX_BWD}


@pytest.mark.parametrize("name", LINEAR)
def test_linear_refusals(name):
    base = LINEAR[name]
    last = B.ERR_WORKSPACE_TOO_SMALL if "ws_bytes" in base else B.ERR_NULL_ARG
    assert call(name, base) == last
    assert call(name, base, dtype=2) == B.ERR_UNSUPPORTED_DTYPE
    assert call(name, base, dtype=-1) == B.ERR_UNSUPPORTED_DTYPE
    for over in (dict(R=-1), dict(R=1 << 31), dict(R=(1 << 31) - (1 << 16) + 1), dict(K=0),
                 dict(K=-64), dict(K=60), dict(K=(1 << 20) + 64), dict(O=0), dict(O=44), dict(O=(1 << 20) + 8), dict(E=0),
                 dict(E=257), dict(off=None), dict(E=256, O=(1 << 17) + 8)):
        assert call(name, base, **over) == B.ERR_BAD_SHAPE, over
    if name.startswith("mx4"):  # whole groups of 32
        assert call(name, base, K=72) == B.ERR_BAD_SHAPE
    for p in ("ldx", "ldy", "lddy", "lddx"):
        if p in base:
            for ld in (40, 68, (1 << 21) + 8, -64):
                assert call(name, base, **{p: ld}) == B.ERR_BAD_SHAPE, (p, ld)
    full = dict(base)
    for p in ("y", "ws_bytes"):
        if p in full:
            full[p] = FAKE
    for p in ("x", "w", "dy", "wq", "y", "dx", "dw", "ws"):
        if p in full and (p != "ws" or "ws_bytes" in full):
            assert call(name, full, **{p: FAKE + 8}) == B.ERR_BAD_ARG, p
    assert call(name, full, off=FAKE + 2) == B.ERR_BAD_ARG
    # one matrix for all rows needs no offsets
    assert call(name, base, off=None, E=1) == last


def test_linear_bwd_pointers():
    need = tm.moe_linear_bwd_workspace_bytes(8, 64, 48, 4)
    assert call("moe_linear_bwd", BWD, ws_bytes=need - 1) == B.ERR_WORKSPACE_TOO_SMALL
    for over in (dict(dx=None, dw=None), dict(w=None), dict(ws=None), dict(dy=None), dict(x=None)):
        assert call("moe_linear_bwd", BWD, ws_bytes=need, **over) == B.ERR_NULL_ARG, over
    # what is not wanted needs no operand: the workspace check is the first to fail
    for over in (dict(dx=None, w=None, lddx=0), dict(dw=None, x=None, ldx=0)):
        assert call("moe_linear_bwd", BWD, **over) == B.ERR_WORKSPACE_TOO_SMALL, over


def test_workspaces():
    f, g = tm.moe_linear_bwd_workspace_bytes, tm.mx4_linear_bwd_workspace_bytes
    for bad in ((-1, 64, 48, 4), (8, 60, 48, 4), (8, 64, 44, 4), (8, 64, 48, 0), (8, 64, 48, 257),
                (8, 0, 48, 4), (8, 64, 0, 4), (1 << 31, 64, 48, 4)):
        assert f(*bad) == 0 and g(*bad) == 0, bad
    assert g(8, 72, 48, 4) == 0 < f(8, 72, 48, 4)
    assert f(0, 64, 48, 4) > 0 and g(0, 64, 48, 4) >= 4 * 64 * 48 * 2
    # few tiles over a long sum: chunks of it, sixteen at most, of 128 elements or a multiple (512)
    assert f(20, 64, 6464, 1) == 13 * 20 * 64 * 4 + 256
    # an average of 4096 rows each, 5120 a part: 6 experts have more, and 12 parts, at most
    assert f(32768, 768, 2432, 8) == 12 * 768 * 2432 * 4 + 256
    # one expert's 114 tiles of 128 x 128: four parts, and a fifth where they do not divide
    assert f(32768, 768, 2432, 1) == 5 * 768 * 2432 * 4 + 256
    assert f(16384, 768, 2432, 17) == 256
    assert f(1 << 20, 8192, 8192, 16) == 256  # parts of more than a gigabyte are not made


def test_mx4_refusals():
    for name, base in (("mx4_pack", PACK), ("mx4_unpack", UNPACK)):
        assert call(name, base) == B.ERR_NULL_ARG
        assert call(name, base, dtype=2) == B.ERR_UNSUPPORTED_DTYPE
        for over in (dict(R=-1), dict(R=1 << 31), dict(C=0), dict(C=60), dict(C=1 << 31),
                     dict(ldx=56), dict(ldx=68)):
            assert call(name, base, **over) == B.ERR_BAD_SHAPE, over
        assert call(name, base, scale=FAKE, x=FAKE + 8) == B.ERR_BAD_ARG
        assert call(name, base, scale=FAKE, q=FAKE + 2) == B.ERR_BAD_ARG
    for rows in (-1, 3):
        assert call("mx4_linear_fwd", MX, rows=rows) == B.ERR_BAD_ARG
    for rows in (1, 2):  # packed rows need their scales; their pitch is their own
        assert call("mx4_linear_fwd", MX, rows=rows, y=FAKE, ldx=0) == B.ERR_NULL_ARG


def test_front_end_refusals():
    x, w = torch.zeros(4, 64), torch.zeros(2, 16, 64)
    off = torch.zeros(3, dtype=torch.int32)
    p = tm.Mx4(torch.zeros(2, 16, 32, dtype=torch.uint8), torch.zeros(2, 16, 2, dtype=torch.uint8))
    for f in (lambda: tm.moe_linear_fwd(x, w, off), lambda: tm.moe_linear_bwd(x, x, w, off),
              lambda: tm.mx4_pack(x), lambda: tm.mx4_unpack(p), lambda: tm.mx4_linear_fwd(x, p, off),
              lambda: tm.mx4_linear_bwd(x, p, off),
              lambda: tm.mx4_linear_fwd(tm.Mx4(p.q[0], p.scale[0]), p, off)):
        with pytest.raises(ValueError, match="no CPU path"):
            f()
    for f in (lambda: tm.mx4_pack([1.0]), lambda: tm.mx4_unpack(p.q), lambda: tm.moe_linear_fwd(1, w)):
        with pytest.raises(TypeError):
            f()


def test_stage_counts():
    from top_moe_layer_amd import block

    assert block._STAGES["moe_linear_bwd"] == B.LINEAR_BWD_STAGES == len(tm.LINEAR_BWD_STAGE_NAMES)
    assert block._STAGES["mx4_linear_bwd"] == B.MX4_BWD_STAGES == len(tm.MX4_BWD_STAGE_NAMES)


# ------------------------------------------------------------ the format's reference
def test_e2m1_ties_and_order():
    mid = (R.E2M1[1:] + R.E2M1[:-1]) / 2
    assert R.to_e2m1(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]  # to the even code
    assert R.to_e2m1(-mid).tolist() == [8, 10, 10, 12, 12, 14, 14]
    assert R.to_e2m1(mid * (1 + 1e-12)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert R.to_e2m1(mid * (1 - 1e-12)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert R.to_e2m1(R.E2M1).tolist() == list(range(8))


def test_mx4_reference():
    x = torch.zeros(6, 40)
    x[0, 3] = 6.0            # 6 * 2^0: nothing is above 6
    x[1, 3] = 6.0000005      # the next scale
    x[2, 3], x[2, 4] = math.inf, 1.0
    x[3, 35] = math.nan
    x[4, 0] = 2.0 ** -149
    x[5, 32], x[5, 33] = -3.0, 0.25
    q, s = R.mx4(x)
    assert q.shape == (6, 20) and s.shape == (6, 2)
    assert s.tolist() == [[127, 0], [128, 0], [255, 0], [0, 255], [0, 0], [0, 126]]
    v = R.from_mx4(q, s)
    assert v[0, 3] == 6.0 and v[1, 3] == 6.0 and v[5, 32] == -3.0 and v[5, 33] == 0.25
    assert torch.isnan(v[2, :32]).all() and not torch.isnan(v[2, 32:]).any()
    assert torch.isnan(v[3, 32:]).all() and (v[4] == 0).all()
    g = torch.Generator().manual_seed(1)
    y = torch.randn(50, 96, generator=g) * torch.exp2(torch.randint(-30, 30, (50, 1), generator=g).float())
    v = R.from_mx4(*R.mx4(y))
    # halfway from 1 to 1.5 times a power of two a value is off by a fifth of itself, the most there
    # is; below 2^e the steps are 2^e / 2
    step = torch.exp2(R.mx4(y)[1].double() - 127).repeat_interleave(32, -1)
    assert bool(((v - y).abs() <= torch.maximum(y.double().abs() / 5, step / 4)).all())
    top = y.abs().reshape(50, 3, 32).amax(-1) / torch.exp2(R.mx4(y)[1].double() - 127)
    assert bool(((top > 3) & (top <= 6)).all())  # the smallest scale


def test_grouped_reference():
    x, w = torch.arange(8.0).reshape(4, 2), torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]]])
    assert R.grouped(x, w, [1, 2]).flatten().tolist() == [0.0, 6.0, 10.0, 0.0]
    assert R.grouped_dw(x[:, :1], x, [1, 2]).tolist() == [[[0.0, 0.0]], [[4 + 16.0, 6 + 20.0]]]


def test_workspace_of_a_dtype():
    f, bf16, fp32 = tm.moe_linear_bwd_workspace_bytes, torch.bfloat16, torch.float32
    # 1024 rows each: parts in fp32 alone, of 1280 rows: 6 experts have more, and 12 parts, at most
    assert f(8192, 2048, 4096, 8, bf16) == 256
    assert f(8192, 2048, 4096, 8, fp32) == 12 * 2048 * 4096 * 4 + 256 == f(8192, 2048, 4096, 8)
    for R, K, O, E in ((0, 64, 48, 4), (20, 64, 6464, 1), (32768, 768, 2432, 8), (16384, 768, 2432, 17),
                       (2400, 72, 136, 8), (1 << 20, 8192, 8192, 16)):
        assert f(R, K, O, E) == max(f(R, K, O, E, bf16), f(R, K, O, E, fp32)) >= 256
    assert f(8, 60, 48, 4, bf16) == f(8, 64, 48, 257, fp32) == 0
    assert B.lib().moe_linear_bwd_dtype_workspace_bytes(8, 64, 48, 4, 2) == 0
    with pytest.raises(TypeError):
        f(8, 64, 48, 4, torch.float16)
    # a call asks for what its dtype needs (and refuses the misaligned workspace behind that check)
    over = dict(R=8192, K=2048, O=4096, E=8, lddy=4096, ldx=2048, lddx=2048, ws=FAKE + 8)
    for dtype, code in ((bf16, B.DTYPE_BF16), (fp32, B.DTYPE_FP32)):
        need = f(8192, 2048, 4096, 8, dtype)
        assert call("moe_linear_bwd", BWD, dtype=code, ws_bytes=need, **over) == B.ERR_BAD_ARG
        assert call("moe_linear_bwd", BWD, dtype=code, ws_bytes=need - 1, **over) == B.ERR_WORKSPACE_TOO_SMALL
