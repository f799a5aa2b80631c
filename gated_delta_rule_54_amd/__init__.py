"""MI355X-native gated delta rule: forward and VJP behind the libgdr C ABI,
with the linear attention with decay, the group norm and the attention layer
(rotary positions, paged cache, windowed attention) that stand beside it.

The kernels are hand-written HIP for gfx950 (csrc/); ``binding`` marshals
torch tensors to the C entry points declared in include/gdr.h.
"""

from .attention import (gdr_attention_backward, gdr_attention_backward_workspace, gdr_attention_forward,
                        gdr_cache_append, gdr_cache_attention, gdr_cache_attention_workspace, gdr_rotary_backward,
                        gdr_rotary_forward)
from .binding import (GdrError, SavedChunks, gdr_backward, gdr_backward_workspace, gdr_calib_copy,
                      gdr_calib_mfma, gdr_forward, gdr_forward_noalloc, gdr_forward_workspace, gdr_keeps_chunks,
                      gdr_profile_enable, gdr_profile_read, lib)
from .linear import (gdr_group_norm_backward, gdr_group_norm_backward_workspace, gdr_group_norm_forward,
                     gdr_linear_backward, gdr_linear_backward_workspace, gdr_linear_forward,
                     gdr_linear_forward_workspace)

__all__ = ["GdrError", "SavedChunks", "gdr_forward", "gdr_forward_noalloc", "gdr_backward", "gdr_forward_workspace",
           "gdr_backward_workspace", "gdr_keeps_chunks", "gdr_profile_enable", "gdr_profile_read",
           "gdr_calib_copy", "gdr_calib_mfma", "gdr_linear_forward", "gdr_linear_backward",
           "gdr_linear_forward_workspace", "gdr_linear_backward_workspace", "gdr_group_norm_forward",
           "gdr_group_norm_backward", "gdr_group_norm_backward_workspace", "gdr_rotary_forward",
           "gdr_rotary_backward", "gdr_cache_append", "gdr_cache_attention", "gdr_cache_attention_workspace",
           "gdr_attention_forward", "gdr_attention_backward", "gdr_attention_backward_workspace", "lib"]
