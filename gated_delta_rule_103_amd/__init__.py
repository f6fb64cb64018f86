"""MI355X-native Kimi Delta Attention (KDA): chunked/varlen prefill and decode.

The compute lives in libkda.so (hand-written HIP kernels for gfx950 behind the
C ABI of include/kda.h); ``kda`` is its ctypes binding, ``linear`` the part for linear attention
without the delta rule, ``serving`` the part for draft trees and the slots of a state pool.
"""
from .kda import (KDAError, gdn_decode, gdn_prefill, gdn_prefill_backward, gdn_recurrent, kda_decode,  # noqa: F401
                  kda_layer_norm, kda_layer_norm_backward, kda_output_gate, kda_output_gate_backward, kda_prefill,
                  kda_prefill_backward, kda_prefill_backward_workspace_size, kda_prefill_noalloc,
                  kda_prefill_snapshots, kda_prefill_workspace_size, kda_recurrent, load_library)
from .linear import (lin_decode, lin_prefill, lin_prefill_backward, lin_prefill_backward_workspace_size,  # noqa: F401
                     lin_prefill_workspace_size, lin_recurrent)
from .serving import (gdn_tree, gdn_tree_accept, kda_slots_acquire, kda_slots_compact, kda_slots_copy,  # noqa: F401
                      kda_slots_release, kda_slots_share, kda_tree, kda_tree_accept, lin_tree, lin_tree_accept)

__all__ = ["kda_prefill", "kda_prefill_noalloc", "kda_prefill_snapshots", "kda_decode", "gdn_prefill", "gdn_decode",
           "kda_recurrent", "gdn_recurrent", "kda_prefill_backward", "gdn_prefill_backward", "kda_output_gate",
           "kda_output_gate_backward", "kda_layer_norm", "kda_layer_norm_backward", "kda_prefill_workspace_size",
           "kda_prefill_backward_workspace_size", "lin_prefill", "lin_prefill_backward", "lin_decode", "lin_recurrent",
           "lin_prefill_workspace_size", "lin_prefill_backward_workspace_size", "kda_tree", "gdn_tree", "lin_tree",
           "kda_tree_accept", "gdn_tree_accept", "lin_tree_accept", "kda_slots_copy", "kda_slots_share",
           "kda_slots_release", "kda_slots_acquire", "kda_slots_compact", "load_library", "KDAError"]
