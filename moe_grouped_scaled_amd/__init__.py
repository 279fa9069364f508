"""MI355X (gfx950) fused MoE expert-MLP hot path: per-row scaled activation + grouped MXFP8 / NVFP4 / MXFP4
block quantization + grouped MX GEMM, behind the C ABI of include/mgs.h.

``_native`` is the ctypes binding (same names as the C entry points); ``expert_mlp`` drives one
expert-MLP training step (FC1 -> scaled activation -> FC2, recompute, delayed wgrad, bias) through it;
``moe`` routes tokens to the experts and back (top-k router, dispatch, combine, their gradients) and holds
``MoELayer``, the layer from router logits to token outputs; ``gated`` has the gated expert block in BF16, forward
and backward, without quantization (``GatedMLP``); ``w4`` serves it with 4-bit weights (``W4GatedMLP``), and
``grad_clip`` has the norm of the gradients and their clipping.
Importing the package loads libmgs.so and raises if it is missing: there is no fallback path.
"""

from . import _native  # noqa: F401
from ._native import (  # noqa: F401
    MgsError,
    QBuf,
    QTensor,
    act_bwd_workspace_bytes,
    act_params,
    grouped_col_sum,
    grouped_gemm_mx,
    grouped_mx_quantize,
    grouped_scaled_act_bwd,
    grouped_scaled_act_fwd,
    qtensor_nbytes,
    quantize_workspace_bytes,
)
from .gated import (  # noqa: F401
    GatedMLP,
    grouped_gated_bwd,
    grouped_gated_bwd_workspace_bytes,
    grouped_gated_fwd,
    grouped_gemm_bf16,
)
from .grad_clip import clip_grad_norm, grad_norm  # noqa: F401
from .moe import (  # noqa: F401
    MoELayer,
    moe_combine,
    moe_combine_bwd,
    moe_dispatch,
    moe_dispatch_bwd,
    moe_route,
    moe_route_bwd,
)
from .w4 import (  # noqa: F401
    W4GatedMLP,
    W4Tensor,
    grouped_gated_w4,
    grouped_gemm_w4,
    w4_pack,
    w4_quantize,
)
