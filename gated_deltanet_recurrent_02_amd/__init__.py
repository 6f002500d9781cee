"""Gated DeltaNet recurrent decode step for MI355X (gfx950).

The compute lives in libgdn.so (hand-written HIP kernels behind the C ABI of include/gdn.h,
include/gdn_linear.h, include/gdn_rotary.h and include/gdn_scan.h); this package holds the ctypes bindings (`decode_step`, `decode_verify`,
`conv_gate_decode`, `prefill`, `prefill_noalloc`, `prefill_workspace_size`, `lowrank_decode_step`,
`lowrank_state`, `state_alloc`; linear attention with a decay for each head:
`linear_attn_decode_step`, `linear_attn_prefill`, `linear_attn_backward`; the norm of a layer's
output: `layer_norm`, `layer_norm_backward`; the rotation of queries and keys by their position and
their norm in every head: `rope`, `rope_backward`, `rope_frequencies`, `qk_norm_rope`,
`qk_norm_rope_backward`; a gated linear recurrence with one value of state a channel:
`gated_scan_decode_step`, `gated_scan_prefill`, `gated_scan_backward`), the in-tree build (`build`), and the seeded
synthetic input generator (`synth`).
"""
from ._binding import (EXPORTS, GDNError, StateBuffer, check, conv_gate_decode, decode_step,
                       decode_verify, lib, lowrank_decode_step, lowrank_state, prefill,
                       prefill_noalloc, prefill_workspace, prefill_workspace_size, state_alloc)
from ._linear import (LINEAR_EXPORTS, layer_norm, layer_norm_backward,
                      layer_norm_backward_workspace_size, linear_attn_backward,
                      linear_attn_backward_workspace_size, linear_attn_decode_step,
                      linear_attn_prefill, linear_attn_prefill_workspace_size)
from ._rotary import (ROTARY_EXPORTS, qk_norm_rope, qk_norm_rope_backward,
                      qk_norm_rope_backward_workspace_size, rope, rope_backward, rope_frequencies)
from ._scan import (GATED_SCAN_CHECKPOINT, SCAN_EXPORTS, gated_scan_backward,
                    gated_scan_backward_workspace_size, gated_scan_decode_step,
                    gated_scan_prefill, gated_scan_prefill_workspace_size)

__all__ = ["EXPORTS", "GATED_SCAN_CHECKPOINT", "GDNError", "LINEAR_EXPORTS", "ROTARY_EXPORTS", "SCAN_EXPORTS", "StateBuffer", "check", "conv_gate_decode",
           "decode_step", "decode_verify", "gated_scan_backward",
           "gated_scan_backward_workspace_size", "gated_scan_decode_step", "gated_scan_prefill",
           "gated_scan_prefill_workspace_size", "layer_norm", "layer_norm_backward",
           "layer_norm_backward_workspace_size", "lib", "linear_attn_backward",
           "linear_attn_backward_workspace_size", "linear_attn_decode_step",
           "linear_attn_prefill", "linear_attn_prefill_workspace_size", "lowrank_decode_step",
           "lowrank_state", "prefill", "prefill_noalloc", "prefill_workspace",
           "prefill_workspace_size", "qk_norm_rope", "qk_norm_rope_backward",
           "qk_norm_rope_backward_workspace_size", "rope", "rope_backward", "rope_frequencies",
           "state_alloc"]
