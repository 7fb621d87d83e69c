"""B200-native (sm_100a) selective state-space scan (S6): a C-ABI CUDA library
(libssm_scan.so, declared in include/ssm_scan.h) and its thin Python binding."""
from .binding import (  # noqa: F401
    ConvSpec,
    FwdOptions,
    SsmError,
    load,
    new_workspace,
    selective_scan_bwd,
    selective_scan_fwd,
    ssm_read_status,
    ssm_selective_scan_bwd,
    ssm_selective_scan_bwd_ex,
    ssm_selective_scan_bwd_workspace_size,
    ssm_selective_scan_fwd,
    ssm_selective_scan_fwd_conv,
    ssm_selective_scan_fwd_noalloc,
    ssm_selective_scan_workspace_size,
    ssm_state_update,
    ssm_state_update_conv,
    ssm_workspace_init,
    status_string,
)
from .gated import (  # noqa: F401
    gated_scan_bwd,
    gated_scan_fwd,
    new_gated_checkpoints,
    new_gated_workspace,
    ssm_gated_bwd_workspace_size,
    ssm_gated_checkpoint_size,
    ssm_gated_scan_bwd,
    ssm_gated_scan_fwd,
    ssm_gated_state_update,
)
from .cache import (  # noqa: F401
    CachePools,
    new_cache_workspace,
    ssm_cache_compact,
    ssm_cache_copy,
    ssm_cache_fork,
    ssm_cache_free,
    ssm_cache_workspace_size,
)
