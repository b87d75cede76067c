"""GB300-native sparse 3-D convolution: indice maps, strided output sets and
implicit-GEMM conv forward / dinput / dfilter, and the layers between convolutions
(group norm with activation, dropout, products grouped by expert; layer norm, rotary
positions, attention within segments, the choice of experts), behind the C ABI of
libspc.so.

``binding`` holds the Python functions, named after the C entry points; the
library is built in-tree by ``build.build()``.
"""

from . import binding  # noqa: F401
from .binding import (  # noqa: F401
    SPC_MAP_SUBM_MIRROR,
    SPC_MAP_TRANSPOSED,
    SPC_PREC_EXACT,
    SPC_PREC_TF32,
    SpcError,
    SpcLibraryMissing,
    check_status,
    new_status,
    spc_build_indice_map,
    spc_conv_dgrad,
    spc_conv_fwd,
    spc_conv_fwd_fused,
    spc_conv_fwd_int8,
    spc_get_wait_limit_ns,
    spc_set_wait_limit_ns,
    SPC_ACT_NONE,
    SPC_ACT_RELU,
    SPC_ACT_SILU,
    spc_row_segments,
    spc_group_norm_fwd,
    spc_group_norm_bwd,
    spc_dropout_fwd,
    spc_dropout_bwd,
    spc_grouped_fwd,
    spc_grouped_dgrad,
    spc_grouped_wgrad,
    SPC_MAX_TOP_K,
    SPC_SCORE_SIGMOID,
    SPC_SCORE_SOFTMAX,
    spc_layer_norm_fwd,
    spc_layer_norm_bwd,
    spc_rope_steps,
    spc_rope_fwd,
    spc_rope_bwd,
    spc_route_fwd,
    spc_route_bwd,
    spc_attention_fwd,
    spc_attention_bwd,
    spc_conv_inverse,
    spc_map_row_order,
    spc_maxpool_fwd,
    spc_maxpool_dgrad,
    spc_conv_wgrad,
    spc_out_shape,
    spc_strided_out_coords,
)
