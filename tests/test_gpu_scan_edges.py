"""The gated linear recurrence's gradients with values that are not finite, with both gates on tensors of more than 2^31 values,
and with gates and rates at their ends on two streams at once."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from scan_ref import CHUNK
from test_gpu_large_offsets import big
from test_gpu_scan import Case, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("coupled", [False, True])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("C", [8, 7])
def test_non_finite_values_stay_in_their_channel_backwards(C, act, coupled):
    B, T = 2, 200
    c = Case(B, T, C, act, "f32", coupled)
    _, d = make(B, T, C, act, 7)
    s0 = c.state.cuda()
    inputs = [*c.inputs, d]

    def grads(x, a, b, d, rate):
        kept = torch.empty(B, -(-T // CHUNK), C, device="cuda")
        gdn.gated_scan_prefill(x, a, b, s0.clone(), rate=rate, checkpoints=kept)
        made = gdn.gated_scan_backward(x, a, b, d, state0=s0, rate=rate, state_grad=True, rate_grad=True)
        given = gdn.gated_scan_backward(x, a, b, d, checkpoints=kept, rate=rate, state_grad=True, rate_grad=True)
        return [t for t in (*made, *given) if t is not None]

    rates = [c.kw["rate"], torch.where(torch.arange(C, device="cuda") == 3, -c.kw["rate"], c.kw["rate"])]
    keep = [j for j in range(C) if j != 3]
    for rate in rates:     # the channel's own rate above and below 0
        clean = grads(*inputs, rate)
        for i, t in enumerate(inputs):
            if t is None:
                continue
            for bad in (float("nan"), float("inf"), -float("inf")):
                put = [v if v is None else v.clone() for v in inputs]
                put[i][0, 100, 3] = bad
                for p, q in zip(grads(*put, rate), clean):
                    assert torch.equal(p[..., keep], q[..., keep])
                    if p.dim() > 1:
                        assert torch.equal(p[1], q[1]) or not q[1].isfinite().all()
                if bad != bad and i == 3:      # the adjoint of every earlier token is a NaN
                    assert grads(*put, rate)[0][0, :101, 3].isnan().all()


def test_two_gates_past_2_31_values():
    B, T, C = 1, 33000, 66000
    assert B * T * C > 2 ** 31
    x, a, b = (big(B, T, C, seed=i) for i in (3, 4, 5))
    rate = torch.rand(C, device="cuda") + 0.1
    s = torch.randn(B, C, device="cuda")
    n = 130
    cut = (slice(None), slice(None), slice(C - n, C))
    part = s[:, C - n:].clone()
    kept = torch.empty(B, -(-T // CHUNK), C, device="cuda")
    o = gdn.gated_scan_prefill(x, a, b, s, rate=rate, checkpoints=kept)
    ref = gdn.gated_scan_prefill(x[cut], a[cut], b[cut], part, rate=rate[-n:].clone())
    # two correct results differ by two half steps of bf16 at most, and by their bars of fp32
    torch.testing.assert_close(o[cut].float(), ref.float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(s[:, C - n:], part, rtol=1e-5, atol=1e-6)
    got = gdn.gated_scan_backward(x, a, b, o, checkpoints=kept, rate=rate)
    part = gdn.gated_scan_backward(x[cut], a[cut], b[cut], o[cut], checkpoints=kept[cut].clone(), rate=rate[-n:].clone())
    for p, q in zip(got[:3], part[:3]):
        torch.testing.assert_close(p[cut].float(), q.float(), rtol=2.0 ** -7, atol=1e-5)


def test_growing_and_forgetting_calls_on_two_streams():
    """Tiles that are walked token by token on one stream, ordinary ones on another, captured and replayed as well."""
    B, T, C = 2, 1500, 96
    x, a, d = (torch.randn(B, T, C, device="cuda") for _ in range(3))
    x[:, :1400] = 0
    calls = [torch.full((C,), -0.3, device="cuda"), torch.full((C,), 3.0, device="cuda")]
    a = a.abs() + 1
    d[:, 100:] = 0

    def work(rate):
        s, kept = torch.zeros(B, C, device="cuda"), torch.empty(B, -(-T // CHUNK), C, device="cuda")
        o = gdn.gated_scan_prefill(x, a, None, s, rate=rate, checkpoints=kept)
        return [o, s, kept, *(t for t in gdn.gated_scan_backward(x, a, None, d, rate=rate, rate_grad=True) if t is not None)]
    alone = [work(r) for r in calls]
    assert all(t.isfinite().all() for w in alone for t in w)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = []
        for st, r in zip(streams, calls):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(work(r))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for u, v in zip(got, alone) for p, q in zip(u, v))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(calls[0])
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, alone[0]))
        work(calls[1])
