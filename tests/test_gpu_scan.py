"""The gated linear recurrence on the GPU against a 64-bit reference token by token (scan_ref.py, where the bars
are derived): types, widths, lengths of zero to many chunks, strides, gates at their ends, gradients, graphs."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from scan_ref import CHUNK, TYPES, Forward, backward, half_step

pytestmark = pytest.mark.gpu


def make(B, T, C, dt, seed, order="dense", std=1.0, shift=0.0):
    """A tensor on the CPU and its copy on the GPU, laid out as `order` says."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, T, C, generator=g) * std + shift).to(TYPES[dt])
    if order == "packed":
        wide = torch.full((B, T, 3 * C), float("nan"), dtype=x.dtype)
        wide[..., C:2 * C] = x
        return x, wide.cuda()[..., C:2 * C]
    if order == "odd":        # off every vector's alignment
        flat = torch.full((x.numel() + 1,), float("nan"), dtype=x.dtype)
        flat[1:] = x.flatten()
        return x, flat.cuda()[1:].view(B, T, C)
    if order == "tbc":
        return x, x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    return x, x.cuda()


def within(got, ref, bar, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    over = ((got - ref).abs() - bar).max().item() if ref.numel() else -1.0
    assert over <= 0, f"{what}: past its bar by {over:.3e}"


class Case:
    """Inputs of a call and their 64-bit reference."""

    def __init__(self, B, T, C, act="f32", state="f32", coupled=False, rate=True, lengths=None, order="dense", shift=-1.0,
                 std=2.0, seed=0, first=True):
        self.act, self.sdt, self.coupled = TYPES[act], TYPES[state], coupled
        self.x, self.dx = make(B, T, C, act, seed + 1, order)
        self.a, self.da = make(B, T, C, act, seed + 2, order, std, shift)
        self.b, self.db = (None, None) if coupled else make(B, T, C, act, seed + 3, order, 1.5)
        g = torch.Generator().manual_seed(seed + 4)
        self.rate = torch.exp(torch.randn(C, generator=g)) if rate else None
        self.state = torch.randn(B, C, generator=g).to(self.sdt) if first else torch.zeros(B, C, dtype=self.sdt)
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
        dbl = lambda t: None if t is None else t.double()  # noqa: E731
        self.args = (dbl(self.x), dbl(self.a), dbl(self.b), dbl(self.rate))
        self.ref = Forward(*self.args, self.state.double(), self.lengths)
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.kw = dict(rate=dev(self.rate), lengths=dev(self.lengths))
        self.inputs = (self.dx, self.da, self.db)

    def check_forward(self, o, state, what, checkpoints=None):
        ref, bar = self.ref.outputs()
        assert o.dtype is self.act
        within(o, ref, bar + half_step(ref, self.act), f"o {what}")
        last, err = self.ref.h[:, -1], self.ref.E[:, -1]
        within(state, last, err + half_step(last, self.sdt), f"state {what}")
        if checkpoints is not None:
            within(checkpoints, *self.ref.kept(), f"checkpoints {what}")

    def check_backward(self, got, d_o, dstate, what):
        ref = backward(self.ref, *self.args, d_o.double(), None if dstate is None else dstate.double())
        names = ("dx", "da", "db", "dstate0", "drate")
        for n, t in zip(names, got):
            if t is None:
                continue
            r, bar = ref[n]
            within(t, r, bar + half_step(r, t.dtype), f"{n} {what}")


def run_all(c, B, T, C, act, order="dense", what=""):
    """decode, prefill with and without checkpoints, backward with and without them, against the reference."""
    s = c.state.cuda()
    o = gdn.gated_scan_decode_step(*c.inputs, s, **c.kw)
    c.check_forward(o, s, f"decode {what}")
    s = c.state.cuda()
    c.check_forward(gdn.gated_scan_prefill(*c.inputs, s, **c.kw), s, f"prefill {what}")
    s = c.state.cuda()
    kept = torch.full((B, -(-T // CHUNK), C), float("nan"), device="cuda")
    c.check_forward(gdn.gated_scan_prefill(*c.inputs, s, checkpoints=kept, **c.kw), s, f"prefill {what}", kept)
    d, dd = make(B, T, C, act, 77, order)
    g = torch.Generator().manual_seed(5)
    dl = torch.randn(B, C, generator=g).to(c.sdt)
    for more in (dict(state0=c.state.cuda()), dict(checkpoints=kept)):
        got = gdn.gated_scan_backward(*c.inputs, dd, dstate=dl.cuda(), state_grad=True, rate_grad=True, **more, **c.kw)
        assert (got[2] is None) == c.coupled
        c.check_backward(got, d, dl, f"{sorted(more)} {what}")


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("act,state", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("B,T,C", [(2, 1, 8), (3, 5, 130), (1, 64, 128), (2, 65, 33), (1, 300, 256), (2, 193, 1), (1, 640, 20)])
def test_every_form(B, T, C, act, state, rate, coupled):
    c = Case(B, T, C, act, state, coupled, rate)
    run_all(c, B, T, C, act, what=f"{B} {T} {C}")


@pytest.mark.parametrize("order", ["packed", "odd", "tbc"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_strides(order, act):
    B, T, C = 3, 150, 64
    c = Case(B, T, C, act, order=order, lengths=[150, 70, 0])
    run_all(c, B, T, C, act, order, order)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,lengths", [(3, [3, 0, 1, 2]), (64, [64, 63, 0, -5]), (130, [130, 64, 65, 1]), (700, [100, 700, 999, 640])])
def test_lengths(T, lengths, act):
    B, C = 4, 70
    c = Case(B, T, C, act, lengths=lengths)
    run_all(c, B, T, C, act, what=str(lengths))
    # what lies past the lengths is not read, and comes back as zeros
    n = c.lengths.clamp(0, T)
    past = torch.arange(T)[None, :] >= n[:, None]
    bad = [t.clone() for t in c.inputs]
    for t in bad:
        t[past.cuda()] = float("nan")
    d = torch.randn(B, T, C, device="cuda").to(c.act)
    d[past.cuda()] = float("inf")
    s = c.state.cuda()
    o = gdn.gated_scan_prefill(*bad, s, **c.kw)
    c.check_forward(o, s, "past")
    for t in gdn.gated_scan_backward(*bad, d, state0=c.state.cuda(), state_grad=True, rate_grad=True, **c.kw):
        assert t.isfinite().all()
        if t.dim() == 3:
            assert not t[past.cuda()].any()


def test_outputs_into_one_packed_tensor():
    B, T, C = 2, 100, 48
    c = Case(B, T, C, "bf16")
    wide = torch.full((B, T, 4 * C), 7.0, device="cuda").bfloat16()
    part = [wide[..., i * C:(i + 1) * C] for i in range(4)]
    s = c.state.cuda()
    assert gdn.gated_scan_prefill(*c.inputs, s, o=part[3], **c.kw) is part[3]
    d, dd = make(B, T, C, "bf16", 8)
    got = gdn.gated_scan_backward(*c.inputs, dd, state0=c.state.cuda(), dx=part[0], da=part[1], db=part[2], **c.kw)
    assert got[0] is part[0]
    c.check_forward(part[3], s, "packed")
    c.check_backward(got, d, None, "packed")
    o = part[3].clone()
    s = c.state.cuda()
    assert torch.equal(gdn.gated_scan_prefill(*c.inputs, s, **c.kw), o)


@pytest.mark.parametrize("coupled", [False, True])
def test_long_memories(coupled):
    """Decays within 2^-20 of 1 over many chunks: what alpha's rounding would lose, step after step."""
    B, T, C = 1, 3000, 64
    c = Case(B, T, C, "f32", coupled=coupled, shift=-13.0, std=1.0)
    run_all(c, B, T, C, "f32")
    c = Case(B, T, C, "bf16", coupled=coupled, shift=-13.0, std=1.0, rate=False)
    run_all(c, B, T, C, "bf16")


def test_gates_at_their_ends():
    """Gates from shut to open, rates of zero, huge and negative ones."""
    B, T, C = 1, 70, 32
    c = Case(B, T, C, "f32", std=30.0, shift=0.0)
    run_all(c, B, T, C, "f32", what="wide gates")
    for value in (0.0, 100.0, 1e-7, -0.01):
        c = Case(B, T, C, "f32")
        c.rate = torch.full((C,), value)
        c.kw["rate"] = c.rate.cuda()
        c.args = (*c.args[:3], c.rate.double())
        c.ref = Forward(*c.args, c.state.double(), None)
        run_all(c, B, T, C, "f32", what=f"rate {value}")
    # a shut token keeps the state bit for bit, an open one forgets it
    x, s = torch.ones(1, 2, 4, device="cuda"), torch.full((1, 4), 3.0, device="cuda")
    a, b = torch.full_like(x, -1e30), torch.full_like(x, -1e30)
    assert torch.equal(gdn.gated_scan_decode_step(x, a, b, s), torch.full_like(x, 3.0))
    a, b = torch.full_like(x, float("inf")), torch.full_like(x, float("inf"))
    assert torch.equal(gdn.gated_scan_prefill(x, a, b, s), torch.ones_like(x)) and torch.equal(s, x[:, 0])


def test_non_finite_values_stay_in_their_channel():
    B, T, C = 2, 200, 8
    c = Case(B, T, C, "f32")
    clean = gdn.gated_scan_prefill(*c.inputs, c.state.cuda(), **c.kw)
    for i in range(3):
        for bad in (float("nan"), float("inf")):
            t = [v.clone() for v in c.inputs]
            t[i][0, 100, 3] = bad
            o = gdn.gated_scan_prefill(*t, c.state.cuda(), **c.kw)
            if bad != bad:
                assert o[0, 100:, 3].isnan().all()
            assert torch.equal(o[0, :64], clean[0, :64]) and torch.equal(o[1], clean[1])
            keep = [j for j in range(C) if j != 3]
            assert torch.equal(o[0][:, keep], clean[0][:, keep])


def test_gradients_against_differences():
    B, T, C = 1, 70, 3
    g = torch.Generator().manual_seed(21)
    x, a, b, d = (torch.randn(B, T, C, generator=g).cuda() for _ in range(4))
    rate, s0 = torch.rand(C, generator=g).cuda() + 0.5, torch.randn(B, C, generator=g).cuda()

    def loss():
        s = s0.clone()
        o = gdn.gated_scan_prefill(x, a, b, s, rate=rate)
        return (o.double() * d.double()).sum().item() + s.double().sum().item()

    got = gdn.gated_scan_backward(x, a, b, d, state0=s0, dstate=torch.ones_like(s0), rate=rate, state_grad=True, rate_grad=True)
    h = 2.0 ** -7
    # central differences: h^2 / 6 of a third derivative (of order 10 here) and rounding 2^-22 |loss terms| / h
    for leaf, grad in zip((x, a, b, s0, rate), got):
        flat, gf = leaf.view(-1), grad.reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 12)):
            old = flat[i].item()
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            assert abs((up - down) / (2 * h) - gf[i].item()) <= 3e-3 * (1 + abs(gf[i].item())), i


def test_no_tokens():
    s = torch.randn(2, 8, device="cuda").bfloat16()
    e = torch.empty(2, 0, 8, device="cuda")
    before = s.clone()
    assert gdn.gated_scan_prefill(e, e, e, s).shape == e.shape and torch.equal(s, before)
    r = torch.ones(8, device="cuda")
    dx, da, db, ds, dr = gdn.gated_scan_backward(e, e, None, e, dstate=s, rate=r, state_grad=True, rate_grad=True)
    assert torch.equal(ds, s) and not dr.any() and db is None
    _, _, _, ds, _ = gdn.gated_scan_backward(e, e, None, e, state0=s, state_grad=True)
    assert ds.dtype is s.dtype and not ds.any()
    e = torch.empty(0, 5, 8, device="cuda")
    *_, dr = gdn.gated_scan_backward(e, e, e, e, rate=r, rate_grad=True)
    assert not dr.any()


def test_decoding_on_after_a_prompt():
    """A prompt in two parts and tokens one by one end where the whole prompt does."""
    B, T, C = 2, 260, 96
    c = Case(B, T, C, "bf16")
    s = c.state.cuda()
    cut = lambda i, j: tuple(t[:, i:j] for t in c.inputs)  # noqa: E731
    parts = [gdn.gated_scan_prefill(*cut(0, 129), s, rate=c.kw["rate"]), gdn.gated_scan_prefill(*cut(129, 256), s, rate=c.kw["rate"])]
    for t in range(256, T):
        parts.append(gdn.gated_scan_decode_step(*cut(t, t + 1), s, rate=c.kw["rate"]))
    c.check_forward(torch.cat(parts, 1), s, "in parts")


@pytest.mark.parametrize("B,T,C,act", [(1, 9000, 200, "bf16"), (40, 400, 1500, "bf16"), (3, 2100, 777, "f16"), (2, 1500, 600, "f32")])
def test_many_tiles(B, T, C, act):
    """More tiles than workgroups run at once, long chains of chunks; the same call gives the same bits."""
    lengths = [T - (T * b) // (B + 1) for b in range(B)]
    c = Case(B, T, C, act, lengths=lengths, std=1.0, shift=-3.0)
    d, dd = make(B, T, C, act, 78)
    runs = []
    for _ in range(2):
        s = c.state.cuda()
        kept = torch.empty(B, -(-T // CHUNK), C, device="cuda")
        o = gdn.gated_scan_prefill(*c.inputs, s, checkpoints=kept, **c.kw)
        made = gdn.gated_scan_backward(*c.inputs, dd, state0=c.state.cuda(), state_grad=True, rate_grad=True, **c.kw)
        with_kept = gdn.gated_scan_backward(*c.inputs, dd, checkpoints=kept, rate_grad=True, **c.kw)
        runs.append([o, s, kept, *made, with_kept[0], with_kept[1], with_kept[2], with_kept[4]])
    assert all(torch.equal(p, q) for p, q in zip(*runs))
    c.check_forward(runs[0][0], runs[0][1], "many", runs[0][2])
    c.check_backward(runs[0][3:8], d, None, "many")
    c.check_backward((*runs[0][8:11], None, runs[0][11]), d, None, "many, kept")


def test_refusals_on_the_device():
    x, s = torch.randn(1, 70, 8, device="cuda"), torch.zeros(1, 8, device="cuda")
    with pytest.raises(TypeError, match="a has dtype"):
        gdn.gated_scan_prefill(x, x.half(), None, s)
    with pytest.raises(ValueError, match="b has shape"):
        gdn.gated_scan_prefill(x, x, x[:, :3], s)
    with pytest.raises(ValueError, match="state has shape"):
        gdn.gated_scan_decode_step(x, x, None, s[0])
    with pytest.raises(ValueError, match="rate has shape"):
        gdn.gated_scan_decode_step(x, x, None, s, rate=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="checkpoints has shape"):
        gdn.gated_scan_prefill(x, x, None, s, checkpoints=torch.empty(1, 3, 8, device="cuda"))
    with pytest.raises(ValueError, match="dense in its last"):
        gdn.gated_scan_prefill(x, torch.randn(1, 8, 70, device="cuda").transpose(1, 2), None, s)
    with pytest.raises(ValueError, match="db is given"):
        gdn.gated_scan_backward(x, x, None, x, db=torch.empty_like(x))
    with pytest.raises(TypeError, match="dstate has dtype"):
        gdn.gated_scan_backward(x, x, None, x, state0=s, dstate=s.half())
    with pytest.raises(gdn.GDNError, match="o overlaps x"):
        gdn.gated_scan_prefill(x, x, None, s, o=x)
    with pytest.raises(gdn.GDNError, match="workspace has"):
        gdn.gated_scan_prefill(x, x, None, s, workspace=torch.empty(4, device="cuda"))


def test_graph_replays():
    B, T, C = 2, 300, 64
    x, a, b, d = (torch.randn(B, T, C, device="cuda").bfloat16() for _ in range(4))
    rate, s0 = torch.rand(C, device="cuda") + 0.5, torch.randn(B, C, device="cuda")

    def work():
        s = s0.clone()
        kept = torch.empty(B, -(-T // CHUNK), C, device="cuda")
        o = gdn.gated_scan_prefill(x, a, b, s, rate=rate, checkpoints=kept)
        o1 = gdn.gated_scan_decode_step(x[:, :1], a[:, :1], b[:, :1], s, rate=rate)
        grads = gdn.gated_scan_backward(x, a, b, d, checkpoints=kept, rate=rate, state_grad=True, rate_grad=True)
        more = gdn.gated_scan_backward(x, a, None, d, state0=s0, rate=rate, rate_grad=True)
        return [t for t in (s, kept, o, o1, *grads, *more) if t is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        x.copy_(torch.randn(B, T, C, device="cuda"))
        s0.add_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, work())), i
