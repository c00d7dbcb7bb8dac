"""GB300 (sm_103a) selective log-prob + GRPO loss forward/backward library.

Python face of the C ABI declared in ``include/grpo_gb300.h``; all compute
runs in the CUDA library ``libgrpo_gb300.so`` built from ``csrc/``.
"""

from ._binding import (  # noqa: F401
    EXPORTED,
    GRPO_ERR_BAD_TOKEN_ID,
    GRPO_ERR_DEVICE_TIMEOUT,
    GRPO_ERR_NONFINITE,
    GRPO_OK,
    NOALLOC_MAX_TOKENS,
    GrpoError,
    GrpoParams,
    GrpoShape,
    alloc_workspace,
    grpo_get_plan,
    grpo_launch_timing_enable,
    grpo_launch_timing_read,
    grpo_logp_fwd,
    grpo_logp_fwd_noalloc,
    grpo_loss_fwd_bwd,
    grpo_read_device_status,
    grpo_selftest_bounded_wait,
    grpo_workspace_size,
    lib,
    make_params,
    make_shape,
    status_string,
)
from ._adamw import (  # noqa: F401
    AdamState,
    AdamW,
    GradNorm,
    alloc_adam_state,
    grpo_grad_norm,
    grpo_grad_norm_workspace_size,
)
from ._glu import (  # noqa: F401
    GluBackward,
    GluForward,
    grpo_glu_bwd,
    grpo_glu_bwd_workspace_size,
    grpo_glu_fwd,
    grpo_glu_wgrad,
    grpo_glu_wgrad_workspace_size,
)
from ._norm_ckpt import (  # noqa: F401
    Checkpoint8,
    NormBackward,
    NormForward,
    alloc_ckpt,
    grpo_ckpt_pack,
    grpo_ckpt_size,
    grpo_ckpt_unpack,
    grpo_ckpt_wgrad,
    grpo_ckpt_wgrad_workspace_size,
    grpo_norm_bwd,
    grpo_norm_fwd,
    grpo_norm_workspace_size,
    grpo_selftest_lose_copy,
)
