"""The gated linear recurrence with states that grow (rates below 0): products of decays past fp32's range over states that are
0 or tiny, where the recurrence itself stays in range, against 64-bit references token by token."""
import math

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from scan_ref import CHUNK, half_step
from scan_relative import Relative, backward
from test_gpu_scan import Case, within

pytestmark = pytest.mark.gpu


def inverse_softplus(y):
    return y + math.log(-math.expm1(-y))


def build(B, T, C, act, coupled, grow, x_scale, x_from, state_scale, lengths=None, seed=60):
    """A Case with rates of -1 in the channels 1 mod 3 and of about 1 elsewhere; there tokens of `grow` (first, end, factor) grow
    by about factor each, the others keep the state; x of x_scale from the token x_from on, 0 before, and states of state_scale."""
    c = Case(B, T, C, act, "f32", coupled, True, lengths=lengths, seed=seed)
    g = torch.Generator().manual_seed(seed + 9)
    grows = torch.arange(C) % 3 == 1
    a, x = c.a.float(), c.x.float()
    a[..., grows] = -60.0
    first, end, factor = grow
    value = inverse_softplus(math.log(factor))
    a[:, first:end, grows] = value * (1 + 0.01 * torch.rand(B, min(end, T) - first, int(grows.sum()), generator=g))
    x[..., grows] *= x_scale
    x[:, :x_from, grows] = 0
    c.state[:, grows] *= state_scale
    c.rate = torch.where(grows, torch.full((C,), -1.0), 0.5 + torch.rand(C, generator=g))
    c.grows = grows
    c.x, c.a = x.to(c.act), a.to(c.act)
    c.dx, c.da = c.x.cuda(), c.a.cuda()
    c.kw["rate"] = c.rate.cuda()
    c.inputs = (c.dx, c.da, c.db)
    c.args = (c.x.double(), c.a.double(), c.args[2], c.rate.double())
    c.ref = Relative(*c.args, c.state.double(), c.lengths)
    return c


def run(c, B, T, C, act, d_scale, d_until, dl_scale):
    """decode, prefill and the gradients against the reference; the channels beside the growing ones give the bits of a call in
    which nothing grows. d_o of d_scale before d_until, 0 after; dstate of dl_scale."""
    g = torch.Generator().manual_seed(3)
    d, dl = torch.randn(B, T, C, generator=g), torch.randn(B, C, generator=g)
    d[..., c.grows] *= d_scale
    d[:, d_until:, c.grows] = 0
    dl[:, c.grows] *= dl_scale
    d = d.to(c.act)
    ref = backward(c.ref, *c.args, d.double(), dl.double())
    tame = torch.where(c.grows.cuda(), torch.ones(C, device="cuda"), c.kw["rate"])
    kept = torch.empty(B, -(-T // CHUNK), C, device="cuda")
    outs = []
    for rate in (c.kw["rate"], tame):
        kw = dict(rate=rate, lengths=c.kw["lengths"])
        s = c.state.cuda()
        o = gdn.gated_scan_prefill(*c.inputs, s, checkpoints=kept, **kw)
        made = gdn.gated_scan_backward(*c.inputs, d.cuda(), state0=c.state.cuda(), dstate=dl.cuda(), state_grad=True,
                                       rate_grad=True, **kw)
        given = gdn.gated_scan_backward(*c.inputs, d.cuda(), checkpoints=kept, dstate=dl.cuda(), state_grad=True,
                                        rate_grad=True, **kw)
        outs.append([o, s, kept.clone(), *(t for t in made if t is not None), *(t for t in given if t is not None)])
        if rate is tame:
            continue
        c.check_forward(o, s, "prefill", kept)
        s = c.state.cuda()
        c.check_forward(gdn.gated_scan_decode_step(*c.inputs, s, **kw), s, "decode")
        for how, got in (("made", made), ("given", given)):
            for name, t in zip(("dx", "da", "db", "dstate0", "drate"), got):
                if t is not None:
                    within(t, ref[name][0], ref[name][1] + half_step(ref[name][0], t.dtype), f"{name} {how}")
    rest = ~c.grows.cuda()
    assert all(torch.equal(p[..., rest], q[..., rest]) for p, q in zip(*outs))


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("B,C", [(1, 40), (1, 33), (3, 70)])
def test_slow_growth_over_many_tiles(B, C, act, coupled):
    """1.24 a token over 1100 tokens, 10^102 in all, over a state of 0 (few chains: groups of tiles)."""
    T = 2000
    c = build(B, T, C, act, coupled, (400, 1500, 1.24), 1.0, 1430, 0.0, None if B == 1 else [T, 1490, 1000])
    assert (c.ref.alpha.log().sum(1) > 200).any()
    run(c, B, T, C, act, 1.0, 430, 0.0)


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("B,T,C,act", [(140, 200, 3, "f32"), (140, 200, 6, "bf16"), (50, 600, 5, "f32"), (1, 60, 12, "f32"),
                                       (1, 200, 12, "bf16"), (1, 1300, 12, "f32"), (1, 1300, 13, "bf16")])
def test_growth_within_a_tile(B, T, C, act, coupled):
    """8 a token over 60 tokens, 10^54 in all, over states, inputs and adjoints of 1e-30."""
    c = build(B, T, C, act, coupled, (0, 60, 8.0), 1e-30, 0, 1e-30)
    run(c, B, T, C, act, 1e-30, T, 1e-30)
    if T > 128:
        c = build(B, T, C, act, coupled, (T - 70, T - 10, 8.0), 1e-30, 0, 1e-30, lengths=[T - i % 7 for i in range(B)])
        run(c, B, T, C, act, 1e-30, T, 1e-30)


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("T", [30, 64, 130, 700, 1300])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_growth_within_a_segment(act, T, coupled):
    """1000 a token over 14 tokens, 10^42 in all, over states, inputs and adjoints of 1e-30 and 0."""
    B, C = 2, 10
    for scale in (1e-30, 0.0):
        for first in (0, T - 16, T // 2 // 16 * 16):
            c = build(B, T, C, act, coupled, (first, min(first + 14, T), 1000.0), scale, 0, scale)
            run(c, B, T, C, act, 1e-30, T, 0.0)


def test_zeros_stay_zeros():
    """Nothing comes of nothing, whatever the decays are."""
    B, T, C = 1, 3000, 24
    z = torch.zeros(B, T, C, device="cuda")
    a, rate = torch.full_like(z, 5.0), torch.full((C,), -20.0, device="cuda")
    for b in (z, None):
        s = torch.zeros(B, C, device="cuda")
        assert not gdn.gated_scan_decode_step(z[:, :70], a[:, :70], None if b is None else b[:, :70], s, rate=rate).any()
        assert not gdn.gated_scan_prefill(z, a, b, s, rate=rate).any() and not s.any()
        got = gdn.gated_scan_backward(z, a, b, z, rate=rate, state_grad=True, rate_grad=True)
        assert not any(t.any() for t in got if t is not None)


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("T,first", [(1, 0), (70, 0), (70, 40), (70, 69), (1300, 700)])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_growth_within_a_token(act, T, first, coupled):
    """10^42 in one token, past fp32's range by itself, over states, inputs and adjoints of 1e-30 and 0."""
    B, C = 2, 10
    for scale in (1e-30, 0.0):
        c = build(B, T, C, act, coupled, (first, first + 1, 1e42), scale, 0, scale)
        run(c, B, T, C, act, 1e-30, T, 0.0)
