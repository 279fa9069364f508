"""MI355X (gfx950) fused MoE expert-MLP hot path: per-row scaled activation + grouped MXFP8 / NVFP4 / MXFP4
block quantization + grouped MX GEMM, behind the C ABI of include/mgs.h.

``_native`` is the ctypes binding (same names as the C entry points); ``expert_mlp`` drives one
expert-MLP training step (FC1 -> scaled activation -> FC2, recompute, delayed wgrad, bias) through it;
``moe`` routes tokens to the experts and back (top-k router, dispatch, combine, their gradients) and holds
``MoELayer``, the layer from router logits to token outputs; ``gated`` has the gated expert block in BF16, forward
and backward, without quantization (``GatedMLP``).
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
from .moe import (  # noqa: F401
    MoELayer,
    moe_combine,
    moe_combine_bwd,
    moe_dispatch,
    moe_dispatch_bwd,
    moe_route,
    moe_route_bwd,
)
