"""MI355X-native gated temporal scan (Mamba2-style), forward and backward.

The compute path is the HIP library `libgscan.so` (hand-written gfx950
kernels behind a C ABI, declared in include/gscan.h); `forward` and
`backward` (and `backward_full`, which adds the input gradients) are thin
ctypes wrappers over it, and `gated_scan` is the same as a
torch.autograd.Function.  `state_scan` is the recurrence with a matrix state
per head, an output per token and sequences of any length (training, prompts,
and `state_scan_step` for single tokens); `qk_norm_rope` makes its queries and
keys.  `embed`, `gated_projection` and `linear_cross_entropy` are what a language
model needs around them: its tokens' embedding, the first half of its
feed-forward blocks, and the loss over its vocabulary.  There is no CPU fallback.
"""
from .binding import (forward, forward_enrich, backward, backward_full,  # noqa: F401
                      backward_workspace_bytes, forward_workspace_bytes,
                      backward_full_workspace_bytes, backward_partials, backward_reduce,
                      batched_cifg_update, bias_grad_reduce, library_path, GScanError)
from . import workloads  # noqa: F401
from .autograd import GatedScanFunction, gated_scan  # noqa: F401
from .embedding import (EmbedFunction, embed, embed_backward,  # noqa: F401
                        embed_backward_workspace_bytes, embed_forward)
from .gated import (GatedProjectionFunction, gated_projection,  # noqa: F401
                               gated_projection_backward, gated_projection_backward_workspace_bytes,
                               gated_projection_forward, gated_projection_forward_workspace_bytes)
from .cross_entropy import (LinearCrossEntropyFunction, linear_cross_entropy,  # noqa: F401
                            linear_cross_entropy_backward,
                            linear_cross_entropy_backward_workspace_bytes, linear_cross_entropy_forward,
                            linear_cross_entropy_forward_workspace_bytes)
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
           "qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_forward", "rotary_frequencies",
           "EmbedFunction", "embed", "embed_backward", "embed_backward_workspace_bytes",
           "embed_forward", "GatedProjectionFunction", "gated_projection", "gated_projection_backward",
           "gated_projection_backward_workspace_bytes", "gated_projection_forward",
           "gated_projection_forward_workspace_bytes",
           "LinearCrossEntropyFunction", "linear_cross_entropy", "linear_cross_entropy_backward",
           "linear_cross_entropy_backward_workspace_bytes", "linear_cross_entropy_forward",
           "linear_cross_entropy_forward_workspace_bytes"]
