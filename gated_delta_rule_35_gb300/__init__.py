"""GB300-native chunked forward of the gated delta rule (Gated DeltaNet).

    from gated_delta_rule_35_gb300 import chunk_fwd
    o, h_final = chunk_fwd(q, k, v, g, beta, scale, h0)

and of the operators around it in a mixing layer: conv_fwd / conv_step, scan_fwd /
scan_step, group_norm; with backward passes, for training: the gated linear recurrence
recur_fwd / recur_step / recur_bwd, layer_norm / layer_norm_bwd, and conv_bwd.

The compute runs in ``lib/libgdn.so`` (hand-written sm_103a kernels behind the
C ABI of ``include/gdn.h``); this package only marshals arguments.
"""
from .native import (GdnError, chunk_fwd, chunk_fwd_host, chunk_fwd_stages, check_device_status,
                     decode_step, problem, workspace_bytes)
from .mixer import (conv_fwd, conv_step, group_norm, scan_fwd, scan_step, scan_workspace_bytes)
from .training import (RECUR_EVERY, conv_bwd, conv_bwd_workspace_bytes, layer_norm, layer_norm_bwd,
                       layer_norm_bwd_workspace_bytes, recur_bwd, recur_bwd_workspace_bytes, recur_fwd,
                       recur_step)

__all__ = ["GdnError", "chunk_fwd", "chunk_fwd_host", "chunk_fwd_stages", "check_device_status",
           "decode_step", "problem", "workspace_bytes", "conv_fwd", "conv_step", "scan_fwd",
           "scan_step", "scan_workspace_bytes", "group_norm", "RECUR_EVERY", "recur_fwd", "recur_step",
           "recur_bwd", "recur_bwd_workspace_bytes", "layer_norm", "layer_norm_bwd",
           "layer_norm_bwd_workspace_bytes", "conv_bwd", "conv_bwd_workspace_bytes"]
