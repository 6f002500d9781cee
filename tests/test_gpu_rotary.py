"""The rotation and the norm of queries and keys on the GPU against 64-bit references (rotary_ref.py, where the
bars are derived): types, vector widths, layouts, strides, lengths, far positions, in place, gradients."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from rotary_ref import TYPES, U, angles, cut, half_step, norm, norm_grads, reach, rotate

pytestmark = pytest.mark.gpu


def make(B, T, H, D, dt, seed, order="dense", std=1.0):
    """A tensor on the CPU and its copy on the GPU with the strides of `order`."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, T, H, D, generator=g) * std).to(TYPES[dt])
    if order == "bhtd":
        y = x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    elif order == "packed":
        wide = torch.full((B, T, 2 * H * D + 3 * D), float("nan"), dtype=x.dtype)
        wide[..., D:D + H * D] = x.flatten(2)
        y = wide.cuda()[..., D:D + H * D].view(B, T, H, D)
    elif order == "odd":        # off every vector's alignment
        flat = torch.full((x.numel() + 1,), float("nan"), dtype=x.dtype)
        flat[1:] = x.flatten()
        y = flat.cuda()[1:].view(B, T, H, D)
    else:
        y = x.cuda()
    return x, y


def within(got, ref, bar, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    over = ((got - ref).abs() - bar).max().item() if ref.numel() else -1.0
    assert over <= 0, f"{what}: past its bar by {over:.3e}"


# B, T, Hq, Hk, D, R: every vector width of both layouts, one unit and several per lane, one token and many, single heads
SHAPES = [(2, 5, 4, 2, 128, 128), (1, 1, 3, 0, 16, 16), (3, 7, 6, 2, 80, 40), (2, 3, 5, 1, 36, 12), (1, 4, 3, 3, 50, 18),
          (2, 2, 2, 1, 33, 32), (1, 3, 2, 1, 256, 64), (1, 2, 1, 1, 511, 510), (1, 2, 2, 2, 512, 512), (2, 3, 1, 1, 2, 2),
          (1, 3, 70, 9, 64, 64), (1, 2, 2, 1, 300, 150), (1, 2, 1, 1, 7, 0), (1, 2, 2, 1, 128, 0)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope_and_its_gradient(shape, dt, interleaved):
    B, T, Hq, Hk, D, R = shape
    f = torch.tensor([0.9 ** i for i in range(R // 2)], dtype=torch.float64)
    g = torch.Generator().manual_seed(D)
    pos = torch.randint(-50, 5000, (B, T), generator=g, dtype=torch.int32)
    theta = angles(pos, f, B, T)
    q, dq = make(B, T, Hq, D, dt, 1)
    k, dk = make(B, T, Hk, D, dt, 2) if Hk else (None, None)
    for fn, transposed in ((gdn.rope, False), (gdn.rope_backward, True)):
        got = fn(dq, dk, f.cuda(), positions=pos.cuda(), interleaved=interleaved, amplitude=1.5)
        for x, y in zip((q, k), got):
            if x is None:
                assert y is None
                continue
            assert y.is_contiguous() and y.dtype is x.dtype
            ref = rotate(x.double(), theta, 1.5, interleaved, transposed)
            size = reach(x.double(), theta, 1.5, interleaved)
            bar = half_step(ref, x.dtype) + 32 * U * size
            bar[..., R:] = 0        # copied
            within(y, ref, bar, f"{fn.__name__} {shape}")


@pytest.mark.parametrize("order", ["bhtd", "packed", "odd"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,R", [(64, 64), (24, 8), (5, 4)])
def test_strides_lengths_and_outputs(order, dt, D, R):
    B, T, Hq, Hk = 3, 6, 5, 2
    f, amp = gdn.rope_frequencies(R)
    lengths = torch.tensor([6, 0, 4], dtype=torch.int32)
    theta = angles(None, f, B, T)
    q, dq = make(B, T, Hq, D, dt, 3, order)
    k, dk = make(B, T, Hk, D, dt, 4, order)
    w = torch.rand(D, dtype=torch.float64) + 0.5
    yq, yk = gdn.rope(dq, dk, f.cuda(), lengths=lengths.cuda())
    out_q, out_k = make(B, T, Hq, D, dt, 5, order)[1], make(B, T, Hk, D, dt, 6, order)[1]
    r = gdn.qk_norm_rope(dq, dk, f.cuda(), lengths=lengths.cuda(), q_weight=w.float().cuda(), q_out=out_q, k_out=out_k)
    assert r[0] is out_q and r[1] is out_k
    for x, y, z, wt in ((q, yq, out_q, w.float().double()), (k, yk, out_k, None)):
        ref = cut(rotate(x.double(), theta, amp, False), lengths)
        size = reach(x.double(), theta, amp, False)
        within(y, ref, half_step(ref, x.dtype) + 32 * U * size, "rope")
        n, _ = norm(x.double(), wt, 1e-6)
        ref = cut(rotate(n, theta, amp, False), lengths)
        within(z, ref, half_step(ref, x.dtype) + 64 * U * reach(n, theta, amp, False), "norm")
    # what lies around the outputs is left as it was
    if order == "packed":
        assert out_q._base[..., :D].isnan().all() and out_q._base[..., D + Hq * D:].isnan().all()
    if order == "odd":
        assert out_q._base[0].isnan()


def test_rows_past_the_lengths_are_not_read():
    B, T, H, D = 2, 5, 3, 32
    f, _ = gdn.rope_frequencies(D)
    q = torch.full((B, T, H, D), float("nan"), device="cuda")
    q[0, :3] = 1.0
    lengths = torch.tensor([3, -7], dtype=torch.int32, device="cuda")
    for y in (*gdn.rope(q, q, f.cuda(), lengths=lengths), *gdn.qk_norm_rope(q, q, f.cuda(), lengths=lengths)):
        assert not y[0, 3:].any() and not y[1].any() and y[0, :3].isfinite().all()
    dq, dk, dwq, dwk = gdn.qk_norm_rope_backward(q, q, q, q, f.cuda(), lengths=lengths, params=True)
    assert dwq.isfinite().all() and dwk.isfinite().all() and not dq[0, 3:].any() and not dk[1].any()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_far_positions(dt):
    """Angles of 2^30 radians and more keep their place in the turn."""
    f = torch.tensor([1.0, 0.73, 1e-4], dtype=torch.float64)
    pos = torch.tensor([[2 ** 31 - 1, 2 ** 30 + 1, -2 ** 31, 12345678]], dtype=torch.int32)
    q, dq = make(1, 4, 2, 8, dt, 7)
    theta = angles(pos, f, 1, 4)
    y, _ = gdn.rope(dq, None, f.cuda(), positions=pos.cuda())
    ref = rotate(q.double(), theta, 1.0, False)
    # |theta| < 2^31: its product and the product with 1 / 2 pi, each off by 2^-53 of 2^31 radians at most, twice that with the constant's own
    bar = half_step(ref, q.dtype) + (32 * U + 3 * 2.0 ** -22) * reach(q.double(), theta, 1.0, False)
    within(y, ref, bar, "far")


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_in_a_packed_projection(interleaved):
    B, T, Hq, Hk, D = 2, 70, 6, 2, 64
    f, _ = gdn.rope_frequencies(32)
    g = torch.Generator().manual_seed(9)
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=g).bfloat16().cuda()
    before = qkv.clone()
    q, k = qkv[..., :Hq * D].view(B, T, Hq, D), qkv[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)
    w = torch.rand(Hq, D, device="cuda"), torch.rand(Hk, D, device="cuda")
    args = dict(interleaved=interleaved, q_weight=w[0], k_weight=w[1])
    eq, ek = gdn.qk_norm_rope(q.contiguous(), k.contiguous(), f.cuda(), **args)
    a, b = gdn.qk_norm_rope(q, k, f.cuda(), q_out=q, k_out=k, **args)
    assert a is q and torch.equal(q, eq) and torch.equal(k, ek)
    assert torch.equal(qkv[..., (Hq + Hk) * D:], before[..., (Hq + Hk) * D:])
    # a gradient over itself
    dq, dk = eq.clone(), ek.clone()
    want = gdn.qk_norm_rope_backward(dq, dk, eq, ek, f.cuda(), **args)
    got = gdn.qk_norm_rope_backward(dq, dk, eq, ek, f.cuda(), q_out=dq, k_out=dk, **args)
    assert got[0] is dq and all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm_and_its_gradients(shape, dt, per_head):
    B, T, Hq, Hk, D, R = shape
    interleaved = (D + per_head) % 2 == 0
    f = torch.tensor([0.8 ** i for i in range(R // 2)], dtype=torch.float64)
    theta = angles(None, f, B, T)
    g = torch.Generator().manual_seed(D)
    sets = []
    for H, seed in ((Hq, 1), (Hk, 2)):
        if H:
            x, y = make(B, T, H, D, dt, seed, std=3.0), make(B, T, H, D, dt, seed + 10)
            w = torch.randn((H, D) if per_head else (D,), generator=g)
            sets.append((x, y, w))
        else:
            sets.append(((None, None), (None, None), None))
    (q, dq, wq), (k, dk, wk) = sets
    kw = dict(interleaved=interleaved, amplitude=0.75, eps=1e-5, q_weight=wq.cuda(), k_weight=None if wk is None else wk.cuda())
    fr = f.cuda() if R else None
    y = gdn.qk_norm_rope(q[1], k[1], fr, **kw)
    grads = gdn.qk_norm_rope_backward(dq[1], dk[1], q[1], k[1], fr, **kw)
    eps = float(torch.tensor(1e-5))
    for i, (x, d, w) in enumerate(sets):
        if x[0] is None:
            assert y[i] is None and grads[i] is None and grads[2 + i] is None
            continue
        n, _ = norm(x[0].double(), w.double(), eps)
        ref = rotate(n, theta, 0.75, interleaved)
        within(y[i], ref, half_step(ref, x[0].dtype) + 64 * U * reach(n, theta, 0.75, interleaved), f"norm {shape}")
        dx, dw, bar_x, bar_w = norm_grads(x[0].double(), d[0].double(), w.double(), eps, theta, 0.75, interleaved, None)
        within(grads[i], dx, half_step(dx, x[0].dtype) + bar_x, f"dx {shape}")
        if not per_head:
            dw, bar_w = dw.sum(0), bar_w.sum(0)
        within(grads[2 + i], dw, bar_w + half_step(dw, torch.float32), f"dw {shape}")


@pytest.mark.parametrize("Hq,Hk,D,R,T", [(48, 16, 128, 128, 3000), (2, 1, 64, 32, 5001), (1, 1, 16, 16, 40000), (3, 1, 40, 12, 2500)])
def test_many_tokens(Hq, Hk, D, R, T):
    """Several tokens a wave, loops over the tokens, every slab of the weights' gradients, ragged."""
    B = 2
    f, _ = gdn.rope_frequencies(R)
    lengths = torch.tensor([T, T // 2 + 3], dtype=torch.int32)
    theta = angles(None, f, B, T)
    kw = dict(lengths=lengths.cuda())
    q, k = make(B, T, Hq, D, "bf16", 1), make(B, T, Hk, D, "bf16", 2)
    dq, dk = make(B, T, Hq, D, "bf16", 3), make(B, T, Hk, D, "bf16", 4)
    y = gdn.qk_norm_rope(q[1], k[1], f.cuda(), **kw)
    z = gdn.rope(q[1], k[1], f.cuda(), **kw)
    grads = gdn.qk_norm_rope_backward(dq[1], dk[1], q[1], k[1], f.cuda(), params=True, **kw)
    for i, (x, d) in enumerate(((q, dq), (k, dk))):
        x, d = x[0].double(), d[0].double()
        ref = cut(rotate(x, theta, 1.0, False), lengths)
        within(z[i], ref, half_step(ref, torch.bfloat16) + 32 * U * reach(x, theta, 1.0, False), "rope")
        n, _ = norm(x, None, 1e-6)
        ref = cut(rotate(n, theta, 1.0, False), lengths)
        within(y[i], ref, half_step(ref, torch.bfloat16) + 64 * U * reach(n, theta, 1.0, False), "norm")
        dx, dw, bar_x, bar_w = norm_grads(x, d, None, 1e-6, theta, 1.0, False, lengths)
        within(grads[i], dx, half_step(dx, torch.bfloat16) + bar_x, "dx")
        within(grads[2 + i], dw.sum(0), bar_w.sum(0) + half_step(dw.sum(0), torch.float32), "dw")


def test_gradients_against_differences():
    B, T, H, D = 1, 3, 2, 12
    f, _ = gdn.rope_frequencies(8)
    g = torch.Generator().manual_seed(11)
    x, d = torch.randn(B, T, H, D, generator=g).cuda(), torch.randn(B, T, H, D, generator=g).cuda()
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()

    def loss(x, w):
        y, _ = gdn.qk_norm_rope(x, None, f.cuda(), q_weight=w, eps=1e-3)
        return (y.double() * d.double()).sum().item()

    dx, _, dw, _ = gdn.qk_norm_rope_backward(d, None, x, None, f.cuda(), q_weight=w, eps=1e-3)
    h = 2.0 ** -7
    # central differences: h^2 / 6 of a third derivative (of order 10 here) and rounding 2^-23 |loss terms| / h
    for at, grad in ((x, dx), (w, dw)):
        flat, gf = at.view(-1), grad.view(-1)
        for i in range(0, flat.numel(), 5):
            old = flat[i].item()
            flat[i] = old + h
            up = loss(x, w)
            flat[i] = old - h
            down = loss(x, w)
            flat[i] = old
            assert abs((up - down) / (2 * h) - gf[i].item()) <= 2e-3 * (1 + abs(gf[i].item())), i


def test_rows_of_zeros_and_optional_outputs():
    q = torch.zeros(1, 2, 3, 32, device="cuda")
    y, none = gdn.qk_norm_rope(q, None)
    assert none is None and not y.any()
    d = torch.randn_like(q)
    dx, dk, dw, dwk = gdn.qk_norm_rope_backward(d, None, q, None, eps=1e-4)
    assert dk is None and dw is None and dwk is None
    torch.testing.assert_close(dx, d * 100.0, rtol=1e-5, atol=0)
    dx2, _, dw, _ = gdn.qk_norm_rope_backward(d, None, q, None, eps=1e-4, params=True)
    assert torch.equal(dx, dx2) and dw.shape == (32,) and not dw.any()
    # no tokens: the weights' gradients are zeros
    e = torch.empty(2, 0, 3, 32, device="cuda")
    _, _, dw, _ = gdn.qk_norm_rope_backward(e, None, e, None, q_weight=torch.ones(3, 32, device="cuda"))
    assert dw.shape == (3, 32) and not dw.any()
    assert gdn.rope(e, e, torch.ones(4, dtype=torch.float64, device="cuda"))[0].shape == e.shape


def test_broadcast_inputs():
    """Inputs may be expanded; their gradients are of the whole shape."""
    x = torch.randn(1, 1, 4, 64, device="cuda").bfloat16().expand(3, 5, 4, 64)
    d = torch.randn(1, 5, 1, 64, device="cuda").bfloat16().expand(3, 5, 4, 64)
    f = gdn.rope_frequencies(64)[0].cuda()
    w = torch.rand(64, device="cuda")
    for fn, args in ((gdn.qk_norm_rope, (x,)), (gdn.qk_norm_rope_backward, (d, None, x))):
        a = fn(*args, None, f, q_weight=w)
        b = fn(*(t if t is None else t.contiguous() for t in args), None, f, q_weight=w)
        assert all(torch.equal(s, t) for s, t in zip(a, b) if t is not None)


def test_refusals_on_the_device():
    f = gdn.rope_frequencies(16)[0].cuda()
    q = torch.randn(1, 2, 2, 32, device="cuda")
    with pytest.raises(TypeError, match="dtype"):
        gdn.rope(q.double(), None, f)
    with pytest.raises(TypeError, match="k has dtype"):
        gdn.rope(q, q.half(), f)
    with pytest.raises(TypeError, match="freqs has dtype"):
        gdn.rope(q, None, f.float())
    with pytest.raises(TypeError, match="positions has dtype"):
        gdn.rope(q, None, f, positions=torch.zeros(1, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="positions has shape"):
        gdn.rope(q, None, f, positions=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="dense in its last"):
        gdn.rope(q.transpose(2, 3).contiguous().transpose(2, 3), None, f)
    with pytest.raises(ValueError, match="k_out"):
        gdn.rope(q, None, f, k_out=q.clone())
    with pytest.raises(ValueError, match="lengths must be on a HIP device"):
        gdn.rope(q, None, f, lengths=torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="q_weight has shape"):
        gdn.qk_norm_rope(q, None, f, q_weight=torch.ones(16, device="cuda"))
    with pytest.raises(ValueError, match="k_weight"):
        gdn.qk_norm_rope(q, None, f, k_weight=torch.ones(32, device="cuda"))
    with pytest.raises(gdn.GDNError, match="R must be"):
        gdn.rope(q, None, gdn.rope_frequencies(34)[0].cuda())
    with pytest.raises(gdn.GDNError, match="overlap each other"):
        gdn.rope(q, None, f, q_out=torch.empty(1, 1, 2, 32, device="cuda").expand(1, 2, 2, 32))
    with pytest.raises(gdn.GDNError, match="q_out overlaps k"):
        gdn.rope(q, q, f, q_out=q)
    with pytest.raises(gdn.GDNError, match="workspace has"):
        gdn.qk_norm_rope_backward(q, None, q, None, f, params=True, workspace=torch.empty(8, device="cuda"))


def test_graph_replays():
    B, T, Hq, Hk, D = 2, 33, 4, 2, 64
    f = gdn.rope_frequencies(D)[0].cuda()
    q, k, dq, dk = (torch.randn(B, T, h, D, device="cuda").bfloat16() for h in (Hq, Hk, Hq, Hk))
    w = torch.rand(D, device="cuda")
    pos = torch.arange(T, device="cuda").expand(B, T).contiguous().int()

    def work():
        a = gdn.qk_norm_rope(q, k, f, positions=pos, q_weight=w, k_weight=w)
        return (*a, *gdn.rope(q, k, f, positions=pos), *gdn.qk_norm_rope_backward(dq, dk, q, k, f, positions=pos, q_weight=w, k_weight=w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(3):
        q.copy_(torch.randn(B, T, Hq, D, device="cuda"))
        pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, work())), i
