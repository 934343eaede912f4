"""GB300-native MXFP4 mixture-of-experts layer (gpt-oss-style MoE block).

The compute path is the CUDA library ``libmoe_mxfp4.so`` (C ABI in
``include/moe_mxfp4.h``); this package only builds it and binds it.
"""

from . import _lib  # noqa: F401
from ._lib import (MOE_ACT_GELU, MOE_ACT_NONE, MOE_ACT_SILU, MOE_ROUTE_GATING_SIGMOID,  # noqa: F401
                   MOE_ROUTE_GATING_SOFTMAX_ALL, MOE_WEIGHTS_DOWN, MOE_WEIGHTS_GATEUP)  # noqa: F401
from .build import build, LIB_PATH  # noqa: F401


def __getattr__(name):
    # torch-facing helpers are imported lazily so the C binding works without torch
    if name in ("MoELayer", "MoELayerBF16", "prepare_weights", "prepare_weights_bf16", "workspace", "route",
                "build_tile_table", "tile_rows", "max_tiles"):
        from . import api
        return getattr(api, name)
    if name in ("block_norm", "block_norm_backward", "BlockNormGrads", "block_norm_8bit", "BlockNorm8", "ffn_forward",
                "ffn_backward", "FfnGrads", "linear_forward", "linear_backward", "LinearGrads", "sort_tokens",
                "sort_tokens_backward", "SortedTokens", "unsort_tokens", "unsort_tokens_backward", "UnsortGrads",
                "route_backward", "dense_status", "MatvecMXFP4"):
        from . import dense
        value = globals()[name] = getattr(dense, name)  # found directly from now on
        return value
    raise AttributeError(name)
