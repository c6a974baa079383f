"""MI355X (gfx950) MoE-layer forward: HIP kernels behind a C ABI (libmoe.so).

The Python side only marshals torch device tensors and the current HIP stream
into the C calls moe_route, moe_schedule and moe_forward; every step of the
layer runs in the library's kernels.
"""

from .api import (MoEBackward, MoELayer, linear_int8, matmul_int8, pack_mxfp8_scales, prepare_backward,  # noqa: F401
                  quantize_int8, quantize_mxfp8, router_for, shape_for, tile_bf16, tile_int8, tile_mxfp8)
