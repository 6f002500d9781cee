"""Gates of the gated linear recurrence over their whole range, forwards and backwards, against 64-bit references."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from scan_ref import CHUNK, Forward, half_step
from scan_relative import Relative, backward
from test_gpu_scan import Case, make, run_all, within

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


def forgetting(B, T, C, act, coupled, rate, seed):
    """Large states, and tokens that forget them: a Case whose x is 1e4 before such tokens and 1e-3 elsewhere."""
    c = Case(B, T, C, act, "f32", coupled, rate, shift=-3.0, std=1.0, seed=seed)
    g = torch.Generator().manual_seed(seed + 9)
    x, a = c.x.float() * 1e-3, c.a.float()
    for t in sorted({0, 1, 15, 16, 17, 31, 63, 64, 65, 100, 128, 150, 191, 199, T - 1}):
        if t < T:
            a[:, t] = 6 + 24 * torch.rand(B, C, generator=g)
            x[:, max(t - 3, 0):max(t - 2, 0)] *= 1e7
    c.state = c.state * 1e4
    c.x, c.a = x.to(c.act), a.to(c.act)
    c.dx, c.da = c.x.cuda(), c.a.cuda()
    if rate:
        c.rate = 0.5 + torch.rand(C, generator=g)
        c.kw["rate"] = c.rate.cuda()
    c.inputs = (c.dx, c.da, c.db)
    c.args = (c.x.double(), c.a.double(), c.args[2], c.rate.double() if rate else None)
    c.ref = Relative(*c.args, c.state.double(), None)
    return c


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C", [(2, 1, 8), (1, 64, 33), (2, 200, 36), (1, 700, 130)])
def test_tokens_that_forget(B, T, C, act, rate, coupled):
    """What a strong token leaves of a large state, and the small input beside it, to fp32's own steps."""
    c = forgetting(B, T, C, act, coupled, rate, 40)
    s = c.state.cuda()
    c.check_forward(gdn.gated_scan_decode_step(*c.inputs, s, **c.kw), s, "decode")
    s = c.state.cuda()
    kept = torch.empty(B, -(-T // CHUNK), C, device="cuda")
    c.check_forward(gdn.gated_scan_prefill(*c.inputs, s, checkpoints=kept, **c.kw), s, "prefill", kept)
    # the adjoint forgets in the same way: a large one behind the last token
    d, dd = make(B, T, C, act, 77)
    d, dd = (d.float() * 1e-3).to(c.act), (dd.float() * 1e-3).to(c.act)
    dl = torch.randn(B, C, generator=torch.Generator().manual_seed(5)) * 1e4
    ref = backward(c.ref, *c.args, d.double(), dl.double())
    for more in (dict(state0=c.state.cuda()), dict(checkpoints=kept)):
        got = gdn.gated_scan_backward(*c.inputs, dd, dstate=dl.cuda(), state_grad=True, rate_grad=True, **more, **c.kw)
        for name, t in zip(("dx", "da", "db", "dstate0", "drate"), got):
            if t is not None:
                within(t, ref[name][0], ref[name][1] + half_step(ref[name][0], t.dtype), f"{name} {sorted(more)}")


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
def test_infinite_gate_forgets_everything(act, coupled):
    """a = infinity is the limit of a large a: alpha 0, and nothing of it in any gradient (0, not 0 times infinity)."""
    B, T, C = 2, 150, 24
    c = Case(B, T, C, act, "f32", coupled, True)
    c.kw["rate"] = 0.5 + torch.rand(C, device="cuda")
    _, d = make(B, T, C, act, 7)
    runs = []
    for open_ in (1e4, INF):
        a = c.da.clone()
        a[:, ::9, ::2] = open_
        s = c.state.cuda()
        o = gdn.gated_scan_prefill(c.dx, a, c.db, s, **c.kw)
        grads = gdn.gated_scan_backward(c.dx, a, c.db, d, state0=c.state.cuda(), state_grad=True, rate_grad=True, **c.kw)
        runs.append([o, s, *(t for t in grads if t is not None)])
        assert all(t.isfinite().all() for t in runs[-1])
    assert all(torch.equal(p, q) for p, q in zip(*runs))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rate_of_zero_keeps_the_state(act):
    """Whatever a is, infinity and fp32's largest values included."""
    x = torch.randn(1, 100, 8, device="cuda").to(torch.float32 if act == "f32" else torch.bfloat16)
    a = torch.randn_like(x) * 100
    a[:, ::3], a[:, 1::7] = INF, 3e38
    s0 = torch.randn(1, 8, device="cuda")
    for call in (gdn.gated_scan_decode_step, gdn.gated_scan_prefill):
        s = s0.clone()
        o = call(x, a, None, s, rate=torch.zeros(8, device="cuda"))
        assert torch.equal(s, s0) and torch.equal(o, s0.to(x.dtype)[:, None].expand_as(o))
