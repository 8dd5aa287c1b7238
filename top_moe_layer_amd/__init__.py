"""MI355X (gfx950) MiniMind FFN / top-k MoE forward and backward.

The compute lives in ``lib/libtopmoe.so`` (hand-written HIP kernels behind the
C ABI of include/topmoe.h).  This package only marshals torch tensors into
that ABI.  Importing it does not load the library; the first call does, and
fails loudly if the library has not been built.
"""
from ._binding import (  # noqa: F401
    DTYPE_BF16,
    DTYPE_FP32,
    DISPATCH_STAGES,
    DISPATCH_STAGE_NAMES,
    FFN_BWD_STAGES,
    FFN_BWD_STAGE_NAMES,
    FFN_STAGES,
    FFN_STAGE_NAMES,
    MOE_BWD_STAGES,
    MOE_BWD_STAGE_NAMES,
    MOE_STAGES,
    MOE_STAGE_NAMES,
    NORM_BWD_STAGES,
    NORM_BWD_STAGE_NAMES,
    RESTORE8_STAGES,
    LINEAR_BWD_STAGES,
    LINEAR_BWD_STAGE_NAMES,
    MX4_BWD_STAGES,
    MX4_BWD_STAGE_NAMES,
    LIB_PATH,
    StageEvents,
    TopmoeError,
    PATH_FIELDS,
    lib,
    moe_fwd_path,
    set_tile_override,
    strerror,
)


def __getattr__(name):
    # torch-level wrappers are imported lazily so that ``import top_moe_layer_amd``
    # stays cheap for tools that only need the raw binding.
    if name in ("ffn_swiglu_fwd", "moe_ffn_fwd", "ffn_workspace_bytes", "moe_workspace_bytes",
                "MoeOutput", "ffn_swiglu_bwd", "moe_ffn_bwd", "ffn_bwd_workspace_bytes",
                "moe_bwd_workspace_bytes", "FfnGrads", "MoeGrads"):
        from . import ops
        return getattr(ops, name)
    if name in ("moe_dispatch_fwd", "moe_dispatch_bwd", "moe_combine_fwd", "moe_combine_bwd",
                "moe_dispatch_workspace_bytes", "block_prenorm_fwd", "block_prenorm_bwd",
                "block_postnorm_fwd", "block_postnorm_bwd", "block_norm_bwd_workspace_bytes",
                "act8_pack", "act8_unpack", "swiglu_act8_fwd", "swiglu_act8_bwd",
                "ffn_keep8_bytes", "moe_keep8_bytes", "ffn_swiglu_keep8", "ffn_swiglu_restore8",
                "moe_ffn_keep8", "moe_ffn_restore8", "Act8", "MoeRows", "CombineGrads",
                "PrenormOutput", "PrenormGrads", "PostnormOutput", "PostnormGrads", "SwigluAct8",
                "SwigluAct8Grads"):
        from . import block
        globals()[name] = v = getattr(block, name)  # found without this function from now on
        return v
    if name in ("moe_linear_fwd", "moe_linear_bwd", "MoeLinearGrads", "Mx4", "mx4_pack",
                "mx4_unpack", "mx4_linear_fwd", "mx4_linear_bwd",
                "moe_linear_bwd_workspace_bytes", "mx4_linear_bwd_workspace_bytes"):
        from . import linear
        globals()[name] = v = getattr(linear, name)
        return v
    if name in ("swiglu_ffn", "moe_ffn", "moe_dispatch", "moe_combine", "block_prenorm",
                "block_postnorm", "swiglu_act8", "moe_linear", "mx4_linear"):
        from . import autograd
        return getattr(autograd, name)
    raise AttributeError(name)
