"""MI355X-native fused GEMM + ReLU: C = ReLU(A @ B) on gfx950 MFMA."""
from .binding import (  # noqa: F401
    gemm_relu,
    gemm_relu_ex,
    gemm_relu_splitk,
    gemm_relu_splitk_noalloc,
    selected_splitk_config,
    gemm_relu_raw,
    selected_config,
    selected_block_config,
    strerror,
    library_path,
    load_library,
    GemmReluError,
    F16,
    BF16,
    B_KN,
    B_NK,
)
from .groups import (  # noqa: F401
    gemm_relu_grouped,
    gemm_relu_grouped_backward,
    gemm_relu_adapters,
    grouped_workspace_bytes,
    grouped_backward_workspace_bytes,
    adapters_workspace_bytes,
    release_workspaces,
)
from .blocks import (  # noqa: F401
    quantize_blocks,
    gemm_relu_blocks,
    gemm_relu_blocks_backward,
    gemm_relu_experts,
    linear_blocks,
    blocks_backward_workspace_bytes,
    experts_workspace_bytes,
)
