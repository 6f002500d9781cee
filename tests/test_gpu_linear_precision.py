"""Linear attention's prompts and gradients in the precision of single tokens, on the GPU: inputs whose large
terms cancel, so that a factor held in fewer bits than fp32's 24 shows in the result, and the gradients
of the training call (no gradient of the states asked for) against 64-bit references (linear_ref.py).

The inputs of the cancelling sums are exact in the tensors' types and few terms are not zero, so the
count of roundings K is small: the bounds are K 2^-24 of the terms' magnitudes and half a step of
the output's type."""
import math

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
import linear_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DIMS = [16, 32, 64, 128]
# 1 + 2^-7 less a little more than half a unit of its 16th bit: in two bf16 parts (16 bits) it becomes 1 + 2^-7
FINE = 1 + 2.0 ** -7 - 2.0 ** -16 + 2.0 ** -23
EVEN = 1 + 2.0 ** -7


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def run_forward(fn, q, k, v, decay, state, act, scale=1.0):
    q, k, v = (t.to(DT[act]).cuda() for t in (q, k, v))
    S = state.cuda()
    o = fn(q, k, v, decay.cuda(), S, scale=scale)
    torch.cuda.synchronize()
    args = (q, k, v, decay, state, scale)
    return o, S, ref.forward(*args), ref.forward_mag(*args)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [7, 8, 70])
def test_state_enters_the_outputs_in_full(T, act, D):
    # 16 columns of the state, FINE and EVEN in turn, with q = 1 and -1: o = 8 (FINE - EVEN)
    print(f"[case] state in outputs T={T} D={D} {act}", flush=True)
    q, k, v = zeros(1, T, 1, D), zeros(1, T, 1, D), zeros(1, T, 1, D)
    state = zeros(1, 1, D, D)
    state[..., 0:16:2], state[..., 1:16:2] = FINE, EVEN
    q[..., 0:16:2], q[..., 1:16:2] = 1.0, -1.0
    o, S, want, mag = run_forward(gdn.linear_attn_prefill, q, k, v, torch.ones(1), state, act)
    assert torch.equal(S.cpu(), state)
    ref.check(o, want[0], mag[0], 16 + 8, "o")  # 16 terms, the factors


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
def test_scores_enter_the_outputs_in_full(act, D):
    # scores FINE and EVEN in turn, v = 1 and -1: every odd token's o is a multiple of FINE - EVEN
    T = 40
    print(f"[case] scores in outputs D={D} {act}", flush=True)
    q, k, v = zeros(1, T, 1, D), zeros(1, T, 1, D), zeros(1, T, 1, D)
    q[..., :4] = 1.0
    k[..., 0], k[..., 1] = 1.0, 2.0 ** -7
    k[:, 0::2, :, 2], k[:, 0::2, :, 3] = -2.0 ** -16, 2.0 ** -23
    v[:, 0::2], v[:, 1::2] = 1.0, -1.0
    o, _, want, mag = run_forward(gdn.linear_attn_prefill, q, k, v, torch.ones(1), zeros(1, 1, D, D), act)
    ref.check(o[:, :8], want[0][:, :8], mag[0][:, :8], 4 + 8 + 4, "o")  # 4 terms a score, 8 tokens, the factors
    ref.check(o, want[0], mag[0], 4 + T + 4, "o of all tokens")


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("where", ["scores", "state"])
def test_products_of_fp16_values_are_whole(where, D):
    # both factors 11 bits long: (1 + 7/1024)^2 against (1 + 7/1024)(1 + 8/1024)
    T, f, e = 8, 1 + 7 / 1024, 1 + 8 / 1024
    print(f"[case] fp16 products in {where} D={D}", flush=True)
    q, k, v, state = zeros(1, T, 1, D), zeros(1, T, 1, D), zeros(1, T, 1, D), zeros(1, 1, D, D)
    if where == "scores":
        q[..., 0] = f
        k[:, 0::2, :, 0], k[:, 1::2, :, 0] = f, e
        v[:, 0::2], v[:, 1::2] = 1.0, -1.0
    else:
        state[..., 0:8:2], state[..., 1:8:2] = f, e
        q[..., 0:8:2], q[..., 1:8:2] = f, -f
    o, _, want, mag = run_forward(gdn.linear_attn_prefill, q, k, v, torch.ones(1), state, "f16")
    ref.check(o, want[0], mag[0], 8 + 8, "o")  # 8 terms, the factors


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [80, 700])
def test_gradients_state_is_summed_in_full(T, act, D):
    # R gains scale and scale (1 + 2^-7) in two columns, late in the sequence; an early token's
    # k = (1 + 2^-7, -1) takes their difference, which is 0. T = 700 splits the sequence.
    print(f"[case] gradients' state T={T} D={D} {act}", flush=True)
    q, k, v, d_o = (zeros(1, T, 1, D) for _ in range(4))
    d_o[:, T - 2], d_o[:, T - 1] = 1.0, EVEN
    q[:, T - 2, :, 0] = 1.0
    q[:, T - 1, :, 1] = 1.0
    k[:, 0, :, 0], k[:, 0, :, 1] = EVEN, -1.0
    args = [t.to(DT[act]).cuda() for t in (q, k, v)] + [torch.ones(1).cuda(), d_o.to(DT[act]).cuda()]
    got = gdn.linear_attn_backward(*args, scale=FINE)
    torch.cuda.synchronize()
    want, mag = (f(*args, None, None, FINE) for f in (ref.backward, ref.backward_mag))
    for name, g, w, m in zip(("dq", "dk", "dv"), got, want, mag):
        ref.check(g, w, m, 8, name)  # two terms, the factors


# 24 ones: the parts' remainders are as large as they get, and all of the value's sign where parts are cut off
ONES = 1 + 2.0 ** -7 - 2.0 ** -23


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("where", ["state", "scores", "update"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_products_of_fp32_values(sign, where, D):
    # one product ONES^2 in each result: its own rounding, the sum of its parts and the factors' roundings
    T = 8
    print(f"[case] fp32 products in {where} D={D} {sign}", flush=True)
    q, k, v, state = zeros(1, T, 1, D), zeros(1, T, 1, D), zeros(1, T, 1, D), zeros(1, 1, D, D)
    if where == "state":
        state[..., 5], q[..., 5] = ONES, sign * ONES
    elif where == "scores":
        q[..., 3], k[:, 0, :, 3], v[:, 0] = ONES, sign * ONES, 1.0
    else:
        v[:, 2], k[:, 2, :, 7] = ONES, sign * ONES
    o, S, want, mag = run_forward(gdn.linear_attn_prefill, q, k, v, torch.ones(1), state, "f32")
    ref.check(o, want[0], mag[0], 4, "o")
    ref.check(S, want[1], mag[1], 4, "state")


def inputs(B, T, H, Hk, D, act, lengths, decay, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = dict(q=unit(r(B, T, Hk, D)), k=unit(r(B, T, Hk, D)), v=r(B, T, H, D), d_o=r(B, T, H, D))
    x = {n: t.to(DT[act]).cuda() for n, t in x.items()}
    x["decay"] = torch.tensor([decay]).expand(H).contiguous().cuda()
    x["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    x["state"] = (0.3 * r(B, H, D, D)).float().cuda()
    return x


LAYOUTS = [(16, 3, 3), (32, 4, 2), (64, 6, 2), (128, 3, 1), (128, 2, 2)]
# the training call over types and head layouts; 700 and 1025 tokens of few heads are split into pieces
TRAINING = [(2, 97, *layout, act, [97, 60], 0.99) for layout in LAYOUTS for act in ("bf16", "f16", "f32")]
TRAINING += [(1, 700, *layout, act, None, 1.0) for layout in LAYOUTS for act in ("bf16", "f16")]
TRAINING += [(2, 1025, 64, 2, 1, "bf16", [1025, 449], 0.995), (1, 1025, 128, 2, 1, "f16", None, 0.9)]


@pytest.mark.parametrize("B,T,D,H,Hk,act,lengths,decay", TRAINING)
def test_gradients_without_the_states(B, T, D, H, Hk, act, lengths, decay):
    what = f"backward without states B={B} T={T} D={D} H={H}/{Hk} {act}"
    print(f"[case] {what}", flush=True)
    x = inputs(B, T, H, Hk, D, act, lengths, decay, T + D)
    scale, s0 = 1 / math.sqrt(D), x["state"] if H != Hk else None
    got = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=s0, scale=scale,
                                   lengths=x["lengths"])
    torch.cuda.synchronize()
    assert got[3] is None and got[4] is None
    args = (x["q"], x["k"], x["v"], x["decay"], x["d_o"], s0, None, scale, x["lengths"])
    want, mag = ref.backward(*args), ref.backward_mag(*args)
    K = ref.attn_roundings(T, D) + H // Hk
    for name, g, w, m in zip(("dq", "dk", "dv"), got, want, mag):
        ref.check(g, w, m, K, f"{what} {name}")
