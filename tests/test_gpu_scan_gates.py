"""Gates of the gated linear recurrence over their whole range, forwards and backwards, against 64-bit references."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from scan_ref import Forward
from test_gpu_scan import Case, make, run_all

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("act,state", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("B,T,C,lengths", [(2, 1, 8, None), (2, 130, 40, [130, 77]), (1, 700, 33, None)])
def test_input_gates_from_shut_to_open(B, T, C, lengths, act, state, rate):
    """b far beyond where e^-|b| is 0, and infinite: beta is 1 or 0 there, forwards and backwards."""
    c = Case(B, T, C, act, state, rate=rate, lengths=lengths)
    b = torch.randn(B, T, C, generator=torch.Generator().manual_seed(9)) * 60
    for i, end in enumerate((86.0, 87.5, 88.0, 89.0, 100.0, 104.0, 1e4, INF)):
        b[:, i::11, i::5] = end
        b[:, i::13, i + 1::7] = -end
    c.b = b.to(c.act)
    c.db = c.b.cuda()
    c.inputs = (c.dx, c.da, c.db)
    c.args = (*c.args[:2], c.b.double(), c.args[3])
    c.ref = Forward(*c.args, c.state.double(), c.lengths)
    run_all(c, B, T, C, act, what="open and shut")


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
def test_open_input_gate_passes_the_gradient_on(act):
    """beta = 1: the last token's dx is d_o, bit for bit."""
    _, x = make(2, 70, 24, act, 1)
    _, d = make(2, 70, 24, act, 2)
    for open_ in (88.0, 90.0, 120.0, 6e4, INF):
        dx, _, db, _, _ = gdn.gated_scan_backward(x, torch.zeros_like(x), torch.full_like(x, open_), d)
        assert torch.equal(dx[:, -1], d[:, -1]), open_
        assert not db[:, -1].any(), open_
