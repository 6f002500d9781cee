"""Linear attention of few heads and long sequences on the GPU: sequences split into pieces (from six chunks of 64
tokens on), over types, head dims and lengths that end in, at and before a piece's edge, against 64-bit references."""
import pytest

import gated_deltanet_recurrent_02_amd as gdn
from test_gpu_linear import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,Hk,D,act,state", [
    (2, 385, 2, 1, 16, "bf16", "bf16"), (2, 450, 1, 1, 32, "f32", "f16"), (2, 513, 2, 2, 64, "bf16", "f16"),
    (1, 390, 3, 1, 128, "f16", "bf16"), (1, 448, 2, 2, 16, "f16", "f32"), (1, 600, 4, 2, 32, "bf16", "f32"),
    (1, 384, 2, 1, 64, "f32", "bf16"), (1, 400, 1, 1, 128, "f32", "f32")])
def test_split_types(B, T, H, Hk, D, act, state):
    x = inputs(B, T, H, Hk, D, act, state, seed=T, lengths=[T - 70 * b for b in range(B)])
    check_forward(gdn.linear_attn_prefill, x, f"split prefill {B} {T} {H}/{Hk} {D} {act} {state}")
    check_backward(x, f"split backward {B} {T} {H}/{Hk} {D} {act} {state}")


@pytest.mark.parametrize("D,act", [(16, "bf16"), (64, "f32"), (128, "bf16")])
def test_split_lengths(D, act):
    # T = 640 in pieces of 128 tokens (prefill, three sweeps of the gradients and the decay's gradient)
    lengths = [0, 1, 127, 128, 129, 512, 513, 640]
    x = inputs(len(lengths), 640, 1, 1, D, act, "f32", lengths=lengths, decay=0.97, seed=D)
    check_forward(gdn.linear_attn_prefill, x, f"split lengths prefill D={D} {act}")
    check_backward(x, f"split lengths backward D={D} {act}")
