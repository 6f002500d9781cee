"""Gated DeltaNet recurrent decode step for MI355X (gfx950).

The compute lives in libgdn.so (hand-written HIP kernels behind the C ABI of include/gdn.h and
include/gdn_linear.h); this package holds the ctypes bindings (`decode_step`, `decode_verify`,
`conv_gate_decode`, `prefill`, `prefill_noalloc`, `prefill_workspace_size`, `lowrank_decode_step`,
`lowrank_state`, `state_alloc`; linear attention with a decay for each head:
`linear_attn_decode_step`, `linear_attn_prefill`, `linear_attn_backward`; the norm of a layer's
output: `layer_norm`, `layer_norm_backward`), the in-tree build (`build`), and the seeded
synthetic input generator (`synth`).
"""
from ._binding import (EXPORTS, GDNError, StateBuffer, check, conv_gate_decode, decode_step,
                       decode_verify, lib, lowrank_decode_step, lowrank_state, prefill,
                       prefill_noalloc, prefill_workspace, prefill_workspace_size, state_alloc)
from ._linear import (LINEAR_EXPORTS, layer_norm, layer_norm_backward,
                      layer_norm_backward_workspace_size, linear_attn_backward,
                      linear_attn_backward_workspace_size, linear_attn_decode_step,
                      linear_attn_prefill, linear_attn_prefill_workspace_size)

__all__ = ["EXPORTS", "GDNError", "LINEAR_EXPORTS", "StateBuffer", "check", "conv_gate_decode",
           "decode_step", "decode_verify", "layer_norm", "layer_norm_backward",
           "layer_norm_backward_workspace_size", "lib", "linear_attn_backward",
           "linear_attn_backward_workspace_size", "linear_attn_decode_step",
           "linear_attn_prefill", "linear_attn_prefill_workspace_size", "lowrank_decode_step",
           "lowrank_state", "prefill", "prefill_noalloc", "prefill_workspace",
           "prefill_workspace_size", "state_alloc"]
