"""Linear attention with a decay for each head on the GPU against 64-bit references (linear_ref.py
derives the bounds): decode, prefill and backward over types, head layouts, lengths and states, and
the calls around them (streams, graphs, padded batches, extreme decays)."""
import math

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
import linear_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def inputs(B, T, H, Hk, D, act="bf16", state="f32", lengths=None, decay=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    a = DT[act]
    if decay is None:
        decay = torch.exp(-torch.exp2(-8.0 * (torch.arange(H) + 1) / H))
    x = dict(q=unit(r(B, T, Hk, D)).to(a), k=unit(r(B, T, Hk, D)).to(a), v=r(B, T, H, D).to(a),
             d_o=r(B, T, H, D).to(a), decay=torch.as_tensor(decay, dtype=torch.float32).expand(H).contiguous(),
             state=(0.3 * r(B, H, D, D)).to(DT[state]), dstate=(0.3 * r(B, H, D, D)).to(DT[state]),
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32), scale=1 / math.sqrt(D))
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def check_forward(fn, x, what):
    _announce(what)
    B, T, H, D = x["v"].shape
    args = (x["q"], x["k"], x["v"], x["decay"], x["state"], x["scale"], x["lengths"])
    want, mag = ref.forward(*args), ref.forward_mag(*args)
    S = x["state"].clone()
    o = fn(x["q"], x["k"], x["v"], x["decay"], S, scale=x["scale"], lengths=x["lengths"])
    torch.cuda.synchronize()
    K = ref.attn_roundings(T, D)
    ref.check(o, want[0], mag[0], K, what + " o", parts=True)
    ref.check(S, want[1], mag[1], K, what + " state")
    return o, S


def check_backward(x, what, states=True, decay_grad=True):
    _announce(what)
    B, T, H, D = x["v"].shape
    s0, ds = (x["state"], x["dstate"]) if states else (None, None)
    args = (x["q"], x["k"], x["v"], x["decay"], x["d_o"], s0, ds, x["scale"], x["lengths"])
    want, mag = ref.backward(*args), ref.backward_mag(*args)
    got = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=s0, dstate=ds,
                                   scale=x["scale"], lengths=x["lengths"], state_grad=True, decay_grad=decay_grad)
    torch.cuda.synchronize()
    K = ref.attn_roundings(T, D) + H // x["q"].shape[2]
    for name, g, w, m in zip(("dq", "dk", "dv", "dstate0"), got, want, mag):
        ref.check(g, w, m, K, f"{what} {name}", parts=name != "dstate0")
    if decay_grad:
        # two chained sums of T tokens and the sums over rows and sequences
        ref.check(got[4], want[4], mag[4], 2 * K + D * B, what + " ddecay")
    else:
        assert got[4] is None
    return got


LAYOUTS = [(16, 3, 3), (32, 4, 2), (64, 6, 2), (128, 3, 1), (128, 2, 2)]


@pytest.mark.parametrize("act,state", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"),
                                       ("f32", "bf16")])
@pytest.mark.parametrize("D,H,Hk", LAYOUTS)
@pytest.mark.parametrize("T", [1, 2, 5])
def test_decode(T, D, H, Hk, act, state):
    x = inputs(3, T, H, Hk, D, act, state, seed=T * D)
    check_forward(gdn.linear_attn_decode_step, x, f"decode T={T} D={D} H={H}/{Hk} {act} {state}")


@pytest.mark.parametrize("act,state", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("D,H,Hk", LAYOUTS)
@pytest.mark.parametrize("T", [1, 15, 17, 64, 65, 130])
def test_prefill(T, D, H, Hk, act, state):
    x = inputs(2, T, H, Hk, D, act, state, seed=T + D)
    check_forward(gdn.linear_attn_prefill, x, f"prefill T={T} D={D} H={H}/{Hk} {act} {state}")


@pytest.mark.parametrize("act", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,H,Hk", LAYOUTS)
@pytest.mark.parametrize("T", [1, 3, 33, 64, 97, 129])
def test_backward(T, D, H, Hk, act):
    x = inputs(2, T, H, Hk, D, act, "f32", seed=T * 3 + D)
    check_backward(x, f"backward T={T} D={D} H={H}/{Hk} {act}", states=T != 33, decay_grad=T != 97)


@pytest.mark.parametrize("state", ["bf16", "f16"])
def test_backward_16_bit_states(state):
    check_backward(inputs(2, 40, 3, 3, 64, "bf16", state, seed=9), f"backward states {state}")


RAGGED = [0, 1, 63, 64, 65, 140, 141, 500]   # 500 and beyond are clamped to T


@pytest.mark.parametrize("D,act", [(64, "bf16"), (128, "bf16"), (32, "f32"), (128, "f16")])
def test_ragged_lengths(D, act):
    T, B = 141, len(RAGGED)
    x = inputs(B, T, 2, 1, D, act, "f32", lengths=RAGGED, seed=D)
    # what lies past a sequence's end is never read: NaN there changes nothing
    for b, n in enumerate(RAGGED):
        for name in ("q", "k", "v", "d_o"):
            x[name][b, min(n, T):] = float("nan")
    clean = dict(x, **{n: torch.nan_to_num(x[n], nan=0.0) for n in ("q", "k", "v", "d_o")})
    for fn in (gdn.linear_attn_prefill, gdn.linear_attn_decode_step):
        o, S = check_forward(fn, clean, f"ragged {fn.__name__} D={D} {act}")
        S2 = x["state"].clone()
        o2 = fn(x["q"], x["k"], x["v"], x["decay"], S2, scale=x["scale"], lengths=x["lengths"])
        assert torch.equal(o, o2) and torch.equal(S, S2)
        assert torch.equal(S[0], x["state"][0]) and not o[0].any() and not o[1, 1:].any()
    got = check_backward(clean, f"ragged backward D={D} {act}")
    again = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=x["state"],
                                     dstate=x["dstate"], scale=x["scale"], lengths=x["lengths"], state_grad=True,
                                     decay_grad=True)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    assert torch.equal(got[3][0], x["dstate"][0]) and not got[0][0].any() and not got[2][1, 1:].any()


def test_negative_lengths_are_empty():
    x = inputs(2, 20, 2, 2, 64, "bf16", "f32", lengths=[-5, 20], seed=1)
    _announce("negative lengths")
    S = x["state"].clone()
    o = gdn.linear_attn_prefill(x["q"], x["k"], x["v"], x["decay"], S, scale=x["scale"], lengths=x["lengths"])
    assert torch.equal(S[0], x["state"][0]) and not o[0].any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1.0, 2.0 ** -20, 1.0 - 2.0 ** -12, 1e-30, -0.5])
def test_extreme_decays(decay, act):
    x = inputs(1, 150, 2, 2, 64, act, "f32", decay=decay, seed=2)
    for fn in (gdn.linear_attn_prefill, gdn.linear_attn_decode_step):
        check_forward(fn, x, f"{fn.__name__} decay={decay} {act}")
    check_backward(x, f"backward decay={decay} {act}")


@pytest.mark.parametrize("B,T,H,Hk,D,act,state", [
    (1, 700, 2, 2, 128, "bf16", "f32"), (1, 1025, 1, 1, 64, "f32", "f32"), (2, 449, 4, 2, 128, "f16", "f32"),
    (2, 300, 2, 1, 16, "bf16", "bf16"), (2, 260, 1, 1, 32, "f32", "f16"), (2, 331, 2, 2, 64, "bf16", "f16"),
    (1, 257, 3, 1, 128, "f16", "bf16")])
def test_long_few_heads(B, T, H, Hk, D, act, state):
    # few heads and many tokens: work split along the sequence
    x = inputs(B, T, H, Hk, D, act, state, seed=T, lengths=[T - 70 * b for b in range(B)])
    check_forward(gdn.linear_attn_prefill, x, f"long prefill {B} {T} {H}/{Hk} {D} {act}")
    check_backward(x, f"long backward {B} {T} {H}/{Hk} {D} {act}")


@pytest.mark.parametrize("B,H", [(40, 16), (90, 48)])
def test_many_heads(B, H):
    x = inputs(B, 70, H, H, 32, "bf16", "f32", seed=B)
    check_forward(gdn.linear_attn_prefill, x, f"prefill {B} x {H} heads")


def test_prefill_then_decode_is_one_run():
    # a prompt, then single tokens, against one prefill of everything (bf16 o: one rounding each)
    x = inputs(2, 90, 3, 3, 128, "bf16", "f32", seed=4)
    _announce("prefill then decode")
    S = x["state"].clone()
    outs = [gdn.linear_attn_prefill(*(x[n][:, :80].contiguous() for n in "qkv"), x["decay"], S, scale=x["scale"])]
    for t in range(80, 90):
        outs.append(gdn.linear_attn_decode_step(*(x[n][:, t:t + 1].contiguous() for n in "qkv"), x["decay"], S,
                                                scale=x["scale"]))
    args = (x["q"], x["k"], x["v"], x["decay"], x["state"], x["scale"])
    want, mag = ref.forward(*args), ref.forward_mag(*args)
    K = ref.attn_roundings(90, 128)
    ref.check(torch.cat(outs, 1), want[0], mag[0], K, "o", parts=True)
    ref.check(S, want[1], mag[1], K, "state")


def test_gradients_against_differences():
    # the directional derivative of the loss sum(o do) + sum(S_T dS) by central differences of the
    # 64-bit forward pass; eps 1e-6 leaves about 1e-9 relative error in fp64
    x = inputs(1, 37, 2, 1, 32, "f32", "f32", seed=7)
    _announce("gradients against differences")
    got = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=x["state"], dstate=x["dstate"],
                                   scale=x["scale"], state_grad=True, decay_grad=True)
    names = ("q", "k", "v", "state", "decay")
    base = {n: x[n].cpu().double() for n in names}
    g = torch.Generator().manual_seed(8)
    for i, n in enumerate(names):
        direction = torch.randn(base[n].shape, generator=g, dtype=torch.float64)

        def loss(e):
            y = dict(base, **{n: base[n] + e * direction})
            o, S = ref.forward(y["q"], y["k"], y["v"], y["decay"], y["state"], x["scale"])
            return float((o * x["d_o"].cpu().double()).sum() + (S * x["dstate"].cpu().double()).sum())

        diff = (loss(1e-6) - loss(-1e-6)) / 2e-6
        grad = got[(0, 1, 2, 3, 4)[i]].cpu().double()
        mine = float((grad * direction).sum())
        size = float((grad.abs() * direction.abs()).sum())
        # fp32 gradients: K roundings each, of sums up to a few times their size
        assert abs(mine - diff) <= 1e-5 * size + 1e-6, f"d{n}: {mine} against {diff}"


@pytest.mark.parametrize("T", [1, 150])
def test_same_bits_twice_and_on_another_stream(T):
    x = inputs(4, T, 6, 3, 128, "bf16", "f32", seed=5, lengths=[T, 1, max(T - 9, 0), 0])
    _announce(f"twice, T={T}")

    def both():
        S = x["state"].clone()
        o = gdn.linear_attn_prefill(x["q"], x["k"], x["v"], x["decay"], S, scale=x["scale"], lengths=x["lengths"])
        grads = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=x["state"],
                                         dstate=x["dstate"], scale=x["scale"], lengths=x["lengths"], state_grad=True,
                                         decay_grad=True)
        return [o, S, *grads]

    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_two_calls_at_once_with_their_own_workspaces():
    xs = [inputs(1, 600, 2, 1, 128, "bf16", "f32", seed=s) for s in (1, 2)]
    _announce("two calls at once")
    n = gdn.linear_attn_backward_workspace_size(1, 600, 2, 1, 128, 128)
    run = lambda x, ws: gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], scale=x["scale"],  # noqa: E731
                                                 decay_grad=True, workspace=ws)
    alone = [run(x, None) for x in xs]
    torch.cuda.synchronize()
    work = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, ws, s in zip(xs, work, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run(x, ws))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for u, v in zip(a, b):
            assert u is v is None or torch.equal(u, v)


@pytest.mark.parametrize("T", [1, 200])
def test_captured_graph_replays(T):
    # prefill (or decode), norm and both backward passes in one graph, replayed on changing inputs
    # with eager work in between
    x = inputs(2, T, 4, 2, 128, "bf16", "f32", seed=6, lengths=[T, max(T - 30, 1)])
    w = torch.rand(4, 128, device="cuda") + 0.5
    _announce(f"graph T={T}")
    fwd = gdn.linear_attn_decode_step if T == 1 else gdn.linear_attn_prefill

    def step(S, first):
        o = fwd(x["q"], x["k"], x["v"], x["decay"], S, scale=x["scale"], lengths=x["lengths"])
        y, mean, rstd = gdn.layer_norm(o, w, None, stats=True)
        do, dw, db = gdn.layer_norm_backward(x["d_o"], o, mean, rstd, w)
        grads = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], do, state0=first, scale=x["scale"],
                                         lengths=x["lengths"], state_grad=True, decay_grad=True)
        return [o, y, mean, rstd, do, dw, db, *grads]

    first = x["state"].clone()
    S = first.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(S, first)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(S, first)
    for k in range(4):
        x["v"].mul_(0.5 if k % 2 else 1.5)
        S.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs] + [S.clone()]
        S2 = first.clone()
        eager = step(S2, first) + [S2]
        torch.cuda.synchronize()
        for a, b in zip(replayed, eager):
            assert torch.equal(a, b), f"replay {k}"


def test_non_finite_values_stay_in_their_head_and_sequence():
    x = inputs(2, 100, 4, 2, 64, "bf16", "f32", seed=3)
    _announce("non-finite")
    clean = [t.clone() for t in (x["q"], x["k"], x["v"], x["d_o"])]
    S0 = x["state"].clone()

    def run():
        S = S0.clone()
        o = gdn.linear_attn_prefill(x["q"], x["k"], x["v"], x["decay"], S, scale=x["scale"])
        g = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], scale=x["scale"])
        return o, S, g[0], g[1], g[2]

    good = run()
    x["v"][0, 50, 1, 3] = float("inf")
    x["d_o"][0, 20, 1, 5] = float("nan")
    bad = run()
    torch.cuda.synchronize()
    for a, b in zip(good, bad):
        assert torch.equal(a[1], b[1])                      # the other sequence
    for i in (0, 4):                                        # the other heads' o and dv
        for h in (0, 2, 3):
            assert torch.equal(good[i][0, :, h], bad[i][0, :, h])
    for i in (2, 3):                                        # the other q/k head's dq and dk
        assert torch.equal(good[i][0, :, 1], bad[i][0, :, 1])
    assert not torch.isfinite(bad[0][0, 50:, 1, 3]).any()   # an infinity in v reaches its own column from its token on


def test_binding_refusals_on_device_tensors():
    x = inputs(1, 4, 2, 2, 32, "bf16", "f32")
    with pytest.raises(ValueError, match="contiguous"):
        gdn.linear_attn_prefill(x["q"].transpose(1, 2).contiguous().transpose(1, 2), x["k"], x["v"], x["decay"], x["state"])
    with pytest.raises(TypeError, match="k has dtype"):
        gdn.linear_attn_prefill(x["q"], x["k"].float(), x["v"], x["decay"], x["state"])
    with pytest.raises(TypeError, match="decay has dtype"):
        gdn.linear_attn_prefill(x["q"], x["k"], x["v"], x["decay"].double(), x["state"])
    with pytest.raises(ValueError, match="decay has shape"):
        gdn.linear_attn_prefill(x["q"], x["k"], x["v"], x["decay"][:1], x["state"])
    with pytest.raises(TypeError, match="lengths has dtype"):
        gdn.linear_attn_decode_step(x["q"], x["k"], x["v"], x["decay"], x["state"],
                                    lengths=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="lengths must be on a HIP device"):
        gdn.linear_attn_decode_step(x["q"], x["k"], x["v"], x["decay"], x["state"], lengths=torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="state has shape"):
        gdn.linear_attn_decode_step(x["q"], x["k"], x["v"], x["decay"], x["state"][:, :1])
    with pytest.raises(TypeError, match="dstate has dtype"):
        gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=x["state"],
                                 dstate=x["dstate"].bfloat16())
    with pytest.raises(gdn.GDNError, match="overlaps"):
        gdn.linear_attn_prefill(x["q"], x["k"], x["v"], x["decay"], x["state"], o=x["v"])
    n = gdn.linear_attn_backward_workspace_size(1, 4, 2, 2, 32, 32)
    with pytest.raises(gdn.GDNError, match="needed"):
        gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"],
                                 workspace=torch.empty(n - 4, dtype=torch.uint8, device="cuda"))


def test_backward_without_tokens():
    x = inputs(2, 0, 3, 3, 32, "bf16", "f32")
    _announce("backward T=0")
    dq, dk, dv, ds, dl = gdn.linear_attn_backward(x["q"], x["k"], x["v"], x["decay"], x["d_o"], state0=x["state"],
                                                  dstate=x["dstate"], state_grad=True, decay_grad=True)
    assert dq.shape == (2, 0, 3, 32) and torch.equal(ds, x["dstate"]) and not dl.any()
    empty = inputs(0, 5, 3, 3, 32, "bf16", "f32")
    dl = gdn.linear_attn_backward(empty["q"], empty["k"], empty["v"], empty["decay"], empty["d_o"], decay_grad=True)[4]
    assert not dl.any()


@pytest.mark.parametrize("act,state", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("D,H,Hk", LAYOUTS)
@pytest.mark.parametrize("T", [7, 8, 9])
def test_shortest_chunked_prompts(T, D, H, Hk, act, state):
    x = inputs(2, T, H, Hk, D, act, state, seed=T + D, lengths=[T, T - 6])
    check_forward(gdn.linear_attn_prefill, x, f"prefill T={T} D={D} H={H}/{Hk} {act} {state}")
    check_backward(x, f"backward T={T} D={D} H={H}/{Hk} {act} {state}")


def test_rows_beyond_32_bit_offsets_go_token_by_token():
    # 64 rows of H * D values may lie further apart than 32 bits reach
    H, D, T = (1 << 19) + 1, 16, 9
    _announce(f"wide rows H={H} D={D} T={T}")
    r = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_o = (r(1, T, H, D) for _ in range(4))
    decay, state = torch.full((H,), 0.75, device="cuda"), 0.3 * torch.randn(1, H, D, D, device="cuda")
    S, S2 = state.clone(), state.clone()
    o = gdn.linear_attn_prefill(q, k, v, decay, S, scale=0.25)
    assert torch.equal(o, gdn.linear_attn_decode_step(q, k, v, decay, S2, scale=0.25)) and torch.equal(S, S2)
    got = gdn.linear_attn_backward(q, k, v, decay, d_o, state0=state, dstate=S, scale=0.25, state_grad=True,
                                   decay_grad=True)
    torch.cuda.synchronize()
    K = ref.attn_roundings(T, D)
    for h in (0, H // 2, H - 1):
        c = lambda t: t[:, :, h:h + 1].contiguous()  # noqa: E731
        s = lambda t: t[:, h:h + 1].contiguous()  # noqa: E731
        args = (c(q), c(k), c(v), decay[h:h + 1], s(state), 0.25, None)
        want, mag = ref.forward(*args), ref.forward_mag(*args)
        ref.check(c(o), want[0], mag[0], K, f"o of head {h}")
        ref.check(s(S), want[1], mag[1], K, f"state of head {h}")
        args = (c(q), c(k), c(v), decay[h:h + 1], c(d_o), s(state), s(S), 0.25, None)
        want, mag = ref.backward(*args), ref.backward_mag(*args)
        for i, name in enumerate(("dq", "dk", "dv")):
            ref.check(c(got[i]), want[i], mag[i], K + 1, f"{name} of head {h}")
        ref.check(s(got[3]), want[3], mag[3], K + 1, f"dstate0 of head {h}")
        ref.check(got[4][h:h + 1], want[4], mag[4], 2 * K + D, f"ddecay of head {h}")


def test_offsets_beyond_32_bits():
    # more than 2^31 values a tensor; a decay of 0.5 forgets all but the last tokens, so the end of the
    # last sequence has a short 64-bit reference (2^-200 of the state before it remains)
    B, T, H, D, n = 3, 120000, 48, 128, 200
    _announce(f"{B * T * H * D} values a tensor")
    q, k, v, d_o = (torch.randn(B, T, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    decay, S = torch.full((H,), 0.5, device="cuda"), torch.zeros(B, H, D, D, device="cuda")
    scale = 1 / math.sqrt(D)
    o = gdn.linear_attn_prefill(q, k, v, decay, S, scale=scale)
    got = gdn.linear_attn_backward(q, k, v, decay, d_o, scale=scale)
    torch.cuda.synchronize()
    K = ref.attn_roundings(T, D)
    for h in (0, H - 1):
        c = lambda t: t[-1:, -n:, h:h + 1].contiguous()  # noqa: E731
        zero = torch.zeros(1, 1, D, D)
        args = (c(q), c(k), c(v), decay[h:h + 1], zero, scale, None)
        want, mag = ref.forward(*args), ref.forward_mag(*args)
        ref.check(c(o)[:, n // 2:], want[0][:, n // 2:], mag[0][:, n // 2:], K, f"o of head {h}", parts=True)
        ref.check(S[-1:, h:h + 1], want[1], mag[1], K, f"state of head {h}")
        args = (c(q), c(k), c(v), decay[h:h + 1], c(d_o), None, None, scale, None)
        want, mag = ref.backward(*args), ref.backward_mag(*args)
        for i, name in enumerate(("dq", "dk", "dv")):
            ref.check(c(got[i])[:, n // 2:], want[i][:, n // 2:], mag[i][:, n // 2:], K + 1, f"{name} of head {h}", parts=True)
