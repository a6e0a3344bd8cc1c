"""MI355X-native gated temporal scan (Mamba2-style), forward and backward.

The compute path is the HIP library `libgscan.so` (hand-written gfx950
kernels behind a C ABI, declared in include/gscan.h); `forward` and
`backward` (and `backward_full`, which adds the input gradients) are thin
ctypes wrappers over it, and `gated_scan` is the same as a
torch.autograd.Function.  `state_scan` is the recurrence with a matrix state
per head, an output per token and sequences of any length (training, prompts,
and `state_scan_step` for single tokens); `qk_norm_rope` makes its queries and
keys.  There is no CPU fallback.
"""
from .binding import (forward, forward_enrich, backward, backward_full,  # noqa: F401
                      backward_workspace_bytes, forward_workspace_bytes,
                      backward_full_workspace_bytes, backward_partials, backward_reduce,
                      batched_cifg_update, bias_grad_reduce, library_path, GScanError)
from . import workloads  # noqa: F401
from .autograd import GatedScanFunction, gated_scan  # noqa: F401
from .matrix_state import (StateScanFunction, state_scan, state_scan_backward,  # noqa: F401
                         state_scan_backward_workspace_bytes, state_scan_forward,
                         state_scan_forward_workspace_bytes, state_scan_step)
from .qk_norm import (QkNormRopeFunction, qk_norm_rope, qk_norm_rope_backward,  # noqa: F401
                      qk_norm_rope_forward, rotary_frequencies)

__all__ = ["forward", "forward_enrich", "backward", "backward_full", "backward_workspace_bytes",
           "forward_workspace_bytes", "backward_full_workspace_bytes", "backward_partials",
           "backward_reduce", "batched_cifg_update", "bias_grad_reduce", "library_path", "GScanError",
           "workloads", "GatedScanFunction", "gated_scan", "StateScanFunction", "state_scan",
           "state_scan_backward", "state_scan_backward_workspace_bytes", "state_scan_forward",
           "state_scan_forward_workspace_bytes", "state_scan_step", "QkNormRopeFunction",
           "qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_forward", "rotary_frequencies"]
