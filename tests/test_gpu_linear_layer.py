"""Linear attention and layer norm together, as a layer trains and serves with them: a ragged prompt,
the norm of every head's output, the gradients back through both, and decoding from the state that the
prompt left. Each step is held to its own bounds (linear_ref.py) on the values the step before gave."""
import math

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
import linear_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("graph", [False, True])
def test_layer_trains_and_serves(act, graph):
    B, T, H, Hk, D, lengths = 3, 150, 4, 2, 64, [150, 70, 0]
    print(f"[case] layer {act} graph={graph}", flush=True)
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(s, generator=g).to(DT[act]).cuda()  # noqa: E731
    q, k, v, dy = r(B, T, Hk, D), r(B, T, Hk, D), r(B, T, H, D), r(B, T, H, D)
    decay = torch.tensor([0.99, 0.9, 0.5, 1.0]).cuda()
    w, b = (1 + 0.2 * torch.randn(H, D, generator=g)).cuda(), torch.randn(H, D, generator=g).cuda()
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    scale = 1 / D
    for i, m in enumerate(lengths):
        dy[i, m:] = 0  # the loss does not see rows past a sequence's end
    first = torch.zeros(B, H, D, D).cuda()
    state = first.clone()

    def layer():
        state.copy_(first)
        o = gdn.linear_attn_prefill(q, k, v, decay, state, scale=scale, lengths=n)
        y, mean, rstd = gdn.layer_norm(o, w, b, stats=True)
        do, dw, db = gdn.layer_norm_backward(dy, o, mean, rstd, w)
        grads = gdn.linear_attn_backward(q, k, v, decay, do, state0=first, scale=scale, lengths=n, decay_grad=True)
        return o, y, mean, rstd, do, dw, db, *grads

    out = layer()
    torch.cuda.synchronize()
    if graph:
        eager = [t if t is None else t.clone() for t in out]
        kept = state.clone()
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            out = layer()
        for _ in range(3):
            recorded.replay()
            torch.randn(1000, device="cuda").sum().item()
            assert torch.equal(state, kept)
            for a, e in zip(out, eager):
                assert (a is None and e is None) or torch.equal(a, e)
    o, y, mean, rstd, do, dw, db, dq, dk, dv, ds, dl = out
    K = ref.attn_roundings(T, D)
    args = (q, k, v, decay, first, scale, n)
    want, mag = ref.forward(*args), ref.forward_mag(*args)
    ref.check(o, want[0], mag[0], K, "o", parts=True)
    ref.check(state, want[1], mag[1], K, "state")
    KN = D / 64 + 32
    wy, _, wr = ref.layer_norm(o, w, b, 1e-5)
    f = o.cpu().double()
    size = (f.abs() + f.abs().mean(-1, keepdim=True)) * wr[..., None]
    ref.check(y, wy, 2 * size * w.cpu().double().abs() + b.cpu().double().abs(), KN, "y")
    want, mag = ref.layer_norm_backward(dy, o, mean, rstd, w)
    ref.check(do, want[0], 2 * mag[0], KN, "do")
    ref.check(dw, want[1], mag[1], B * T + 32, "dweight")
    ref.check(db, want[2], mag[2], B * T + 32, "dbias")
    args = (q, k, v, decay, do, first, None, scale, n)
    want, mag = ref.backward(*args), ref.backward_mag(*args)
    for name, a, x, m in zip(("dq", "dk", "dv"), (dq, dk, dv), want, mag):
        ref.check(a, x, m, K + H // Hk, name, parts=True)
    ref.check(dl, want[4], mag[4], 2 * K + D * B, "ddecay")
    # two new tokens of every sequence from the state that the prompt left
    q2, k2, v2 = r(B, 2, Hk, D), r(B, 2, Hk, D), r(B, 2, H, D)
    args = (q2, k2, v2, decay, state, scale, None)
    want, mag = ref.forward(*args), ref.forward_mag(*args)
    S = state.clone()
    o2 = gdn.linear_attn_decode_step(q2, k2, v2, decay, S, scale=scale)
    torch.cuda.synchronize()
    ref.check(o2, want[0], mag[0], ref.attn_roundings(2, D), "decoded o")
    ref.check(S, want[1], mag[1], ref.attn_roundings(2, D), "decoded state")
