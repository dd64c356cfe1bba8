"""MI355X (gfx950) routed Mixture-of-Experts layer, the norms around its block and 4-bit experts.

The compute path is libmoe.so (hand-written HIP kernels behind a C ABI, see
include/moe.h); `binding` marshals torch device tensors into it and
`workloads` draws the seeded synthetic inputs.
"""
from . import binding, workloads  # noqa: F401
from .binding import (moe_combine, moe_grouped_ffn, moe_layer_forward, moe_permute,  # noqa: F401
                      moe_route, moe_block_norm, moe_block_norm_backward,
                      moe_w4_grouped_ffn, moe_w4_matvec, moe_w4_pack, moe_w4_quantize, BlockNorm, BlockNormBackward,
                      LayerForward, MoEError, W4GroupedFfn, W4Matvec, W4Quantize, W4Weights)
