"""The rotation, the norm of queries and keys and the gated recurrence as they are used together with what was there: one
layer from a packed projection (norm and rotation in place, linear attention, the gated recurrence on its output, the
layer norm of every head), its gradients, decoding on token by token, graph replays, and calls on two streams at once."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn

pytestmark = pytest.mark.gpu

B, T, H, Hk, D = 2, 150, 4, 2, 32
# Of six stages each is off by at most 2^-17 of the magnitudes that it adds up (the bars of their own tests, in fp32), which
# here are at most 16 times the results'; the layer norm divides by standard deviations of more than 1/4: 6 * 16 * 4 * 2^-17.
BAR = 6 * 16 * 4 * 2.0 ** -17


class Layer:
    def __init__(self, seed=0, dtype=torch.float32):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.cols = (H + 2 * Hk) * D      # q, k, and the first half of v
        self.x = n(B, T, self.cols).to(dtype)
        self.v = n(B, T, H, D).to(dtype)
        self.a, self.b = (n(B, T, H * D) - 1).to(dtype), n(B, T, H * D).to(dtype)
        self.wq, self.wk = (1 + 0.1 * n(D)) * D ** -0.5, (1 + 0.1 * n(Hk, D)[0]) * D ** -0.5
        self.freqs, self.amp = gdn.rope_frequencies(D // 2, scaling="yarn", factor=4.0, original_length=64)
        self.decay = 1 - torch.exp2(-3 - torch.arange(H) / 2.0)
        self.rate = torch.exp(0.5 * n(H * D))
        self.w, self.bias = 1 + 0.1 * n(H, D), 0.1 * n(H, D)
        self.S0, self.h0 = 0.3 * n(B, H, D, D), n(B, H * D)
        self.dy = n(B, T, H, D)
        self.pos = (torch.arange(T)[None] + torch.tensor([[7], [1000]])).int()

    def reference(self):
        """y and the gradients of x, v, a, b, wq, wk, rate in 64 bits, token by token."""
        leaves = {n: getattr(self, n).double().requires_grad_() for n in ("x", "v", "a", "b", "wq", "wk", "rate")}
        x, v, a, b, wq, wk, rate = leaves.values()
        theta = (self.pos.double()[..., None] * self.freqs)[:, :, None]
        c, s = torch.cos(theta) * self.amp, torch.sin(theta) * self.amp

        def heads(z, w):
            z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * w
            r = D // 4
            p, q, rest = z[..., :r], z[..., r:2 * r], z[..., 2 * r:]
            return torch.cat([p * c - q * s, p * s + q * c, rest], -1)
        q = heads(x[..., :H * D].reshape(B, T, H, D), wq)
        k = heads(x[..., H * D:(H + Hk) * D].reshape(B, T, Hk, D), wk)
        q = q.reshape(B, T, Hk, H // Hk, D).mean(3)     # one q a k head, as linear attention shares them
        q, k = (z.repeat_interleave(H // Hk, 2) for z in (q, k))
        S, h, rows = self.S0.double(), self.h0.double(), []
        soft = torch.logaddexp(a, torch.zeros_like(a))
        for t in range(T):
            S = self.decay.double()[:, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
            o = (S * q[:, t, :, None, :]).sum(-1).reshape(B, H * D)
            h = torch.exp(-rate * soft[:, t]) * h + torch.sigmoid(b[:, t]) * o
            rows.append(h)
        h = torch.stack(rows, 1).reshape(B, T, H, D)
        m = h - h.mean(-1, keepdim=True)
        y = m * torch.rsqrt((m * m).mean(-1, keepdim=True) + 1e-5) * self.w.double() + self.bias.double()
        grads = torch.autograd.grad((y * self.dy.double()).sum(), list(leaves.values()))
        return y.detach(), dict(zip(leaves, grads))


def forward(L, c, S, h, kept=None, t0=0, t1=T, step=False):
    """The layer on tokens t0..t1 with the package; returns what a backward pass needs too."""
    x = c["x"][:, t0:t1].clone()
    n = t1 - t0
    q, k = x[..., :H * D].view(B, n, H, D), x[..., H * D:(H + Hk) * D].view(B, n, Hk, D)
    raw_q, raw_k = q.clone(), k.clone()
    pos = c["pos"][:, t0:t1].contiguous()
    how = dict(positions=pos, amplitude=L.amp, q_weight=c["wq"], k_weight=c["wk"])
    gdn.qk_norm_rope(q, k, c["freqs"], q_out=q, k_out=k, **how)       # in place in the packed tensor
    qm = q.reshape(B, n, Hk, H // Hk, D).mean(3).to(q.dtype)
    kc, v = k.contiguous(), c["v"][:, t0:t1].contiguous()
    attn = gdn.linear_attn_decode_step if step else gdn.linear_attn_prefill
    o = attn(qm, kc, v, c["decay"], S)
    a, b = c["a"][:, t0:t1], c["b"][:, t0:t1]
    if step:
        r = gdn.gated_scan_decode_step(o.view(B, n, -1), a, b, h, rate=c["rate"])
    else:
        r = gdn.gated_scan_prefill(o.view(B, n, -1), a, b, h, rate=c["rate"], checkpoints=kept)
    y, mean, rstd = gdn.layer_norm(r.view(B, n, H, D), c["w"], c["bias"], stats=True)
    return y, dict(raw_q=raw_q, raw_k=raw_k, how=how, qm=qm, kc=kc, v=v, o=o, r=r, mean=mean, rstd=rstd)


def on_device(L):
    return {n: v.cuda() for n, v in vars(L).items() if isinstance(v, torch.Tensor)}


def backward(L, c, s, kept):
    dr, _, _ = gdn.layer_norm_backward(c["dy"].to(s["r"].dtype), s["r"].view(B, T, H, D), s["mean"], s["rstd"], c["w"])
    do, da, db, _, drate = gdn.gated_scan_backward(s["o"].view(B, T, -1), c["a"], c["b"], dr.view(B, T, -1),
                                                   checkpoints=kept, rate=c["rate"], rate_grad=True)
    dqm, dk, dv, _, _ = gdn.linear_attn_backward(s["qm"], s["kc"], s["v"], c["decay"], do.view(B, T, H, D), state0=c["S0"])
    dq = (dqm / (H // Hk)).repeat_interleave(H // Hk, 2)
    gx = torch.zeros_like(c["x"])      # the gradients of q and k go straight into the packed one
    gq, gk = gx[..., :H * D].view(B, T, H, D), gx[..., H * D:(H + Hk) * D].view(B, T, Hk, D)
    _, _, dwq, dwk = gdn.qk_norm_rope_backward(dq, dk, s["raw_q"], s["raw_k"], c["freqs"], q_out=gq, k_out=gk, **s["how"])
    return dict(x=gx, v=dv, a=da, b=db, wq=dwq, wk=dwk, rate=drate)


def close(got, ref, bar, what):
    err = (got.double().cpu() - ref).abs().max().item() / ref.abs().max().item()
    assert err <= bar, f"{what}: {err:.3e} > {bar:.3e}"


def test_layer_and_its_gradients():
    L = Layer()
    ref, grads = L.reference()
    c = on_device(L)
    kept = torch.empty(B, -(-T // gdn.GATED_SCAN_CHECKPOINT), H * D, device="cuda")
    y, s = forward(L, c, c["S0"].clone(), c["h0"].clone(), kept)
    close(y, ref, BAR, "y")
    for n, g in backward(L, c, s, kept).items():
        close(g, grads[n], 4 * BAR, n)     # two passes through the stages, and their products


def test_prompt_then_tokens():
    L = Layer(1)
    ref, _ = L.reference()
    c = on_device(L)
    S, h = c["S0"].clone(), c["h0"].clone()
    rows = [forward(L, c, S, h, t0=0, t1=100)[0], forward(L, c, S, h, t0=100, t1=140)[0]]
    for t in range(140, T):
        rows.append(forward(L, c, S, h, t0=t, t1=t + 1, step=True)[0])
    close(torch.cat(rows, 1), ref, BAR, "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_in_16_bits(dtype):
    L = Layer(2, dtype)
    ref, _ = L.reference()
    c = on_device(L)
    y, _ = forward(L, c, c["S0"].clone(), c["h0"].clone())
    # four roundings to 16 bits on the way (half a step each), with the factors of BAR
    close(y, ref, 4 * 16 * 4 * torch.finfo(dtype).eps / 2, "y")


def test_graph_replays_of_the_layer():
    L = Layer(3, torch.bfloat16)
    c = on_device(L)
    kept = torch.empty(B, -(-T // gdn.GATED_SCAN_CHECKPOINT), H * D, device="cuda")

    def work():
        y, s = forward(L, c, c["S0"].clone(), c["h0"].clone(), kept)
        return [y, *backward(L, c, s, kept).values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(3):
        c["x"].copy_(torch.randn(B, T, L.cols, device="cuda"))
        c["a"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, work())), i


def test_two_streams_at_once():
    """Calls that pass states between their tiles, in flight together on two streams with workspaces of their own."""
    cases = []
    for seed, (b, t, ch) in enumerate([(4, 2000, 512), (1, 6000, 256)]):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, a, gb, d = (torch.randn(b, t, ch, generator=g, device="cuda").bfloat16() for _ in range(4))
        cases.append((x, a, gb, d, torch.rand(ch, generator=g, device="cuda"), torch.randn(b, ch, generator=g, device="cuda")))

    def work(x, a, gb, d, rate, s0):
        s = s0.clone()
        o = gdn.gated_scan_prefill(x, a, gb, s, rate=rate)
        return (o, s, *gdn.gated_scan_backward(x, a, gb, d, state0=s0, rate=rate, state_grad=True, rate_grad=True))
    want = [work(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [[], []]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append(work(*cases[i]))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for r in got[i] for p, q in zip(r, want[i]))
