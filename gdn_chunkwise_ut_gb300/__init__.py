"""kkt_solve for GB300: the chunk-local UT transform of Gated DeltaNet prefill.

    from gdn_chunkwise_ut_gb300 import kkt_solve_fwd
    T, W, U = kkt_solve_fwd(k, v, beta, C=64)            # k, v bf16 [B,T,H,128] on cuda
    o, S = gdn_chunk_state_fwd(q, k, W, U, C=64)         # the chunk recurrence that consumes W, U

and the operators that serve a layer around it (include/gdn_layer.h): gdn_prep_fwd, gdn_recurrent_fwd,
add_rms_norm_fwd, gated_rms_norm_fwd, gdn_state_copy.

The computation runs in libkkt.so (hand-written CUDA for sm_103a, C ABI in
include/kkt.h); this package only marshals torch tensors.
"""
from .api import (  # noqa: F401
    HostRunner,
    chunk_gated_delta_rule,
    device_status,
    gdn_chunk_state_fwd,
    host_workspace_bytes,
    kkt_solve_fwd,
    kkt_solve_fwd_host,
    select_kernel,
)
from .layer import (  # noqa: F401
    add_rms_norm_fwd,
    gated_rms_norm_fwd,
    gdn_prep_fwd,
    gdn_recurrent_fwd,
    gdn_state_copy,
)
from .pool import SlotTable, StatePool  # noqa: F401
from ._lib import KktError  # noqa: F401

__all__ = ["kkt_solve_fwd", "kkt_solve_fwd_host", "host_workspace_bytes", "gdn_chunk_state_fwd",
           "chunk_gated_delta_rule", "gdn_recurrent_fwd", "gdn_prep_fwd", "add_rms_norm_fwd", "gated_rms_norm_fwd",
           "gdn_state_copy", "SlotTable", "StatePool", "device_status", "select_kernel", "HostRunner", "KktError"]
