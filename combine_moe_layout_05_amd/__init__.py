"""MI355X (gfx950) MoE token routing layout, dispatch and combine (layout and
dispatch also fused into two launches: MoeDispatcher.layout_dispatch), their
backward, and the expert step between them (grouped GEMMs driven by the
device-side offsets): one linear map per expert, or the gated feed-forward
block with its backward; weights in bf16 or in 4 bits, rows in bf16 or, for
the forward products, in 4 bits. Before them the router (route_topk); for the
few tokens of a decoding step the whole layer in two launches (moe_layer).

The compute lives in libmoe_layout.so (hand-written HIP kernels behind the C
ABI of include/moe.h); this package is its thin Python binding.
"""
from .moe import (  # noqa: F401
    Dispatched, Layout, MoeDispatcher, Mxfp4ExpertWeights, Mxfp4Rows, TiledExpertWeights,
    ceil_div, grouped_gemm, layout_noalloc, num_max_tokens_infer, num_max_tokens_pretrain, round_up4,
    tile_expert_weights, validate_num_max,
)
from ._lib import MoeError, load  # noqa: F401
from .experts import (  # noqa: F401
    dequantize_mxfp4, gated_grouped_gemm, gated_grouped_gemm_backward,
    grouped_gemm_backward_input, grouped_gemm_backward_weight, grouped_gemm_forward,
    mxfp4_expert_weights, quantize_mxfp4,
)
from .autograd import MoeTokenDispatcher, expert_ffn  # noqa: F401
from .router import Routing, route_topk, route_topk_backward  # noqa: F401
from .layer import moe_layer  # noqa: F401
