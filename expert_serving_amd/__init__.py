"""MI355X (gfx950) MoE-layer forward: router, dispatch, grouped SwiGLU FFN, combine.

The compute path is the HIP library `libmoe_mi355x.so` behind the C ABI in
`include/moe_mi355x.h`; `abi` binds it with ctypes.  PyTorch only supplies
device memory and streams.
"""

from . import abi  # noqa: F401
from .abi import (make_block, make_shape, moe_block_forward, moe_block_forward_int8, moe_combine,  # noqa: F401
                  moe_combine_norm, moe_dispatch, moe_grouped_ffn, moe_grouped_ffn_int8, moe_grouped_gemm_int8,
                  moe_layer_forward, moe_norm, moe_quantize_int8, moe_read_device_flags, moe_route_biased,
                  moe_route_topk, moe_workspace_size)
