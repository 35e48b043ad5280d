"""GB300 (sm_103a) latent-MoE output tail.

    out[t, h] = sum_l rms_norm(sum_p routed[p, t, :], g, eps)[l] * W[h, l]
                + sum_p shared[p, t, h]

The computation runs in the CUDA library built from ``csrc/`` and exposed
through the C ABI in ``include/latent_tail.h``; ``binding`` is the thin ctypes
layer over it, and ``block`` the same for the operators around the tail (expert
dispatch and combine, 4-bit expert products, fused residual norms) and ``experts`` for
the bf16 experts with their gradients and for activations in 8 bits. Importing this package does not load the library; the first
call does, and fails loudly if it was not built.
"""

from .binding import (  # noqa: F401
    LatentTailError,
    Status,
    forward,
    forward_host,
    latent_tail_check,
    latent_tail_forward,
    latent_tail_forward_cols,
    latent_tail_forward_host,
    latent_tail_norm,
    latent_tail_project_cols,
    latent_tail_status_string,
    latent_tail_host_workspace_size,
    latent_tail_workspace_size,
    library_path,
    load_library,
)
from .block import (  # noqa: F401
    Dispatched,
    combine,
    combine_backward,
    dispatch,
    dispatch_workspace_size,
    expert_matvec4,
    quantize4,
    residual_norm,
    residual_norm_backward,
    residual_norm_backward_workspace_size,
)
from .experts import (  # noqa: F401
    Checkpoint8,
    dequantize8,
    expert_gated,
    expert_gated_backward,
    expert_gated_backward_workspace_size,
    expert_matmul,
    expert_matmul_backward,
    quantize8,
)
