"""MI355X-native Kimi Delta Attention (KDA): chunked/varlen prefill and decode.

The compute lives in libkda.so (hand-written HIP kernels for gfx950 behind the
C ABI of include/kda.h); ``kda`` is its ctypes binding.
"""
from .kda import (KDAError, gdn_decode, gdn_prefill, gdn_prefill_backward, gdn_recurrent, kda_decode,  # noqa: F401
                  kda_layer_norm, kda_layer_norm_backward, kda_output_gate, kda_output_gate_backward, kda_prefill,
                  kda_prefill_backward, kda_prefill_backward_workspace_size, kda_prefill_noalloc,
                  kda_prefill_snapshots, kda_prefill_workspace_size, kda_recurrent, load_library)

__all__ = ["kda_prefill", "kda_prefill_noalloc", "kda_prefill_snapshots", "kda_decode", "gdn_prefill", "gdn_decode",
           "kda_recurrent", "gdn_recurrent", "kda_prefill_backward", "gdn_prefill_backward", "kda_output_gate",
           "kda_output_gate_backward", "kda_layer_norm", "kda_layer_norm_backward", "kda_prefill_workspace_size",
           "kda_prefill_backward_workspace_size", "load_library", "KDAError"]
