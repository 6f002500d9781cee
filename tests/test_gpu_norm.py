"""Layer norm forward and backward on the GPU against 64-bit references (linear_ref.py derives the
bounds), over types, widths, groups and the calls around them."""
import math

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from gated_deltanet_recurrent_02_amd import _linear
import linear_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = ref.U


def make(shape, dtype, per_head, seed=0, affine=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    ps = shape[-2:] if per_head else shape[-1:]
    x = dict(x=(0.7 * r(*shape) + 0.3).to(DT[dtype]), dy=r(*shape).to(DT[dtype]),
             weight=(1 + 0.2 * r(*ps)).float() if affine else None, bias=(0.1 * r(*ps)).float() if affine else None)
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def check(x, what, eps=1e-5, per_head=False):
    print(f"[case] {what}", flush=True)
    C, rows = x["x"].shape[-1], x["x"].numel() // x["x"].shape[-1]
    K = C / 64 + 32
    y, mean, rstd = gdn.layer_norm(x["x"], x["weight"], x["bias"], eps=eps, stats=True)
    dx, dw, db = gdn.layer_norm_backward(x["dy"], x["x"], mean, rstd, x["weight"], params=True)
    torch.cuda.synchronize()
    wy, wm, wr = ref.layer_norm(x["x"], x["weight"], x["bias"], eps)
    f = x["x"].cpu().double()
    a = lambda t, d: d if t is None else t.cpu().double().abs()  # noqa: E731
    # n = (x - m) r: m is off by K roundings of mean |x|, r by half the variance's K roundings
    size = (f.abs() + f.abs().mean(-1, keepdim=True)) * wr[..., None]
    ref.check(mean, wm, f.abs().mean(-1), K, what + " mean")
    ref.check(rstd, wr, wr * (1 + (f.abs().mean(-1) * wr) ** 2 * K * U), K, what + " rstd")
    ref.check(y, wy, 2 * size * a(x["weight"], 1.0) + a(x["bias"], 0.0), K, what + " y")
    want, mag = ref.layer_norm_backward(x["dy"], x["x"], mean, rstd, x["weight"])
    # each mean's sum may be off by K roundings, and n's two operations by three
    ref.check(dx, want[0], 2 * mag[0], K, what + " dx")
    ref.check(dw, want[1], mag[1], rows + 32, what + " dweight")
    ref.check(db, want[2], mag[2], rows + 32, what + " dbias")
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", [1, 2, 7, 16, 64, 65, 128, 250, 512, 513, 1000, 1024, 2048, 4099, 6144, 8191, 16384, 20000])
def test_widths(C, dtype):
    check(make((5, C), dtype, False, seed=C), f"norm C={C} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 3, 16), (2, 9, 5, 32), (7, 48, 64), (3, 33, 6, 128), (300, 2, 24), (5, 3, 1032)])
def test_per_head(shape, dtype):
    check(make(shape, dtype, True, seed=sum(shape)), f"per head {shape} {dtype}")


@pytest.mark.parametrize("rows,C", [(1, 128), (2, 96), (3, 256), (63, 40), (1025, 128), (4097, 72), (2500, 1536)])
def test_rows(rows, C):
    check(make((rows, C), "bf16", False, seed=rows), f"norm rows={rows} C={C}")


def test_without_affine():
    x = make((40, 200), "f32", False, seed=1, affine=False)
    check(x, "no affine")
    print("[case] no affine, per head", flush=True)
    y = gdn.layer_norm(x["x"])
    dx, dw, db = gdn.layer_norm_backward(x["dy"], x["x"], *gdn.layer_norm(x["x"], stats=True)[1:])
    assert dw is None and db is None and torch.isfinite(dx).all() and y.shape == x["x"].shape


def test_weight_without_bias_and_bias_without_weight():
    x = make((33, 4, 96), "f32", True, seed=2)
    check(dict(x, bias=None), "no bias")
    print("[case] bias alone", flush=True)
    y = gdn.layer_norm(x["x"], None, x["bias"])
    want, _, _ = ref.layer_norm(x["x"], None, x["bias"], 1e-5)
    assert float((y.cpu().double() - want).abs().max()) < 1e-5


def test_in_place_and_over_dy():
    x = make((50, 1000), "bf16", False, seed=3)
    y, mean, rstd, dx, dw, db = check(x, "in place")
    buf = x["x"].clone()
    assert gdn.layer_norm(buf, x["weight"], x["bias"], y=buf) is buf
    assert torch.equal(buf, y)
    # the C ABI also takes dx over dy
    over, w2, b2 = x["dy"].clone(), torch.empty_like(dw), torch.empty_like(db)
    n = gdn.layer_norm_backward_workspace_size(50, 1, 1000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    gdn.check(_linear._lib().gdn_layer_norm_backward(50, 1, 1000, p(over), p(x["x"]), 1, p(x["weight"]), p(mean), p(rstd),
                                                     p(over), p(w2), p(b2), p(ws), n,
                                                     torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(over, dx) and torch.equal(w2, dw) and torch.equal(b2, db)


def test_constant_rows_large_offsets_and_tiny_values():
    print("[case] constant rows", flush=True)
    x = torch.full((3, 300), 5.0, device="cuda")
    y, mean, rstd = gdn.layer_norm(x, stats=True)
    assert torch.equal(mean, torch.full_like(mean, 5.0)) and not y.any()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))
    x = make((4, 640), "f32", False, seed=5)
    x["x"] += 300.0                       # the mean is 400 times the spread
    check(x, "large offset")
    x = make((4, 640), "f32", False, seed=6)
    x["x"] *= 1e-12
    check(x, "tiny values", eps=1e-30)


def test_non_finite_rows_stay_alone():
    x = make((6, 4, 128), "bf16", True, seed=7)
    print("[case] non-finite rows", flush=True)
    y, mean, rstd = gdn.layer_norm(x["x"], x["weight"], x["bias"], stats=True)
    x["x"][2, 1, 5] = float("nan")
    x["x"][4, 3, 0] = float("inf")
    y2, m2, r2 = gdn.layer_norm(x["x"], x["weight"], x["bias"], stats=True)
    same = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    same[2, 1] = same[4, 3] = False
    assert torch.equal(y[same], y2[same]) and torch.equal(mean[same], m2[same])
    assert not torch.isfinite(y2[2, 1]).any() and not torch.isfinite(y2[4, 3]).all()


def test_no_rows():
    x = torch.empty(0, 4, 32, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(4, 32, device="cuda")
    y, mean, rstd = gdn.layer_norm(x, w, stats=True)
    assert y.shape == x.shape and mean.shape == (0, 4)
    dx, dw, db = gdn.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == x.shape and not dw.any() and not db.any()


def test_gradients_against_differences():
    x = make((3, 2, 45), "f32", True, seed=8)
    print("[case] differences", flush=True)
    _, mean, rstd = gdn.layer_norm(x["x"], x["weight"], x["bias"], stats=True)
    got = gdn.layer_norm_backward(x["dy"], x["x"], mean, rstd, x["weight"])
    base = {n: x[n].cpu().double() for n in ("x", "weight", "bias")}
    g = torch.Generator().manual_seed(9)
    for n, grad in zip(("x", "weight", "bias"), got):
        d = torch.randn(base[n].shape, generator=g, dtype=torch.float64)

        def loss(e):
            z = dict(base, **{n: base[n] + e * d})
            return float((ref.layer_norm(z["x"], z["weight"], z["bias"], 1e-5)[0] * x["dy"].cpu().double()).sum())

        diff = (loss(1e-6) - loss(-1e-6)) / 2e-6
        grad = grad.cpu().double()
        assert abs(float((grad * d).sum()) - diff) <= 1e-5 * float((grad.abs() * d.abs()).sum()) + 1e-6, n


def test_same_bits_twice():
    x = make((3000, 4, 128), "bf16", True, seed=10)
    a, b = check(x, "twice (1)"), check(x, "twice (2)")
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_binding_refusals_on_device_tensors():
    x = make((4, 6, 32), "bf16", True)
    with pytest.raises(ValueError, match="weight has shape"):
        gdn.layer_norm(x["x"], x["weight"][:2])
    with pytest.raises(TypeError, match="bias has dtype"):
        gdn.layer_norm(x["x"], x["weight"], x["bias"].bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        gdn.layer_norm(x["x"].transpose(0, 1))
    with pytest.raises(ValueError, match="y has shape"):
        gdn.layer_norm(x["x"], y=x["x"][:2])
    with pytest.raises(ValueError, match="mean has shape"):
        gdn.layer_norm_backward(x["dy"], x["x"], torch.zeros(4, device="cuda"), torch.zeros(4, 6, device="cuda"))
    with pytest.raises(gdn.GDNError, match="eps"):
        gdn.layer_norm(x["x"], eps=-1.0)


@pytest.mark.parametrize("rows,C", [(70000, 64), (3000, 4500)])
def test_parameter_gradients_over_many_slabs(rows, C):
    check(make((rows, C), "bf16", False, seed=rows), f"slabs rows={rows} C={C}")


def test_affine_of_more_than_2_to_27_values():
    G, C = 16400, 8200
    print(f"[case] affine G={G} C={C}", flush=True)
    x = torch.randn(1, G, C, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(1, G, C, device="cuda", dtype=torch.bfloat16)
    weight = torch.full((G, C), 2.0, device="cuda")
    y, mean, rstd = gdn.layer_norm(x, weight, stats=True)
    dx, dw, db = gdn.layer_norm_backward(dy, x, mean, rstd, weight, params=True)
    torch.cuda.synchronize()
    assert torch.equal(db, dy[0].float())  # one row of every group: the sum is the value
    for g in (0, G // 2, G - 1):
        want, mag = ref.layer_norm_backward(dy[:, g], x[:, g], mean[:, g], rstd[:, g], weight[g])
        ref.check(dw[g], want[1], mag[1], 33, f"dweight of group {g}")
        ref.check(dx[:, g], want[0], 2 * mag[0], C / 64 + 32, f"dx of group {g}")


def test_offsets_beyond_32_bits():
    rows, C, n = 17_000_000, 128, 40
    print(f"[case] {rows * C} values", flush=True)
    x, dy = (torch.randn(rows, C, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    weight, bias = torch.full((C,), 1.5, device="cuda"), torch.full((C,), -0.5, device="cuda")
    y, mean, rstd = gdn.layer_norm(x, weight, bias, stats=True)
    dx, _, db = gdn.layer_norm_backward(dy, x, mean, rstd, weight)
    torch.cuda.synchronize()
    K = C / 64 + 32
    for part in (slice(0, n), slice(rows - n, rows)):
        wy, wm, wr = ref.layer_norm(x[part], weight, bias, 1e-5)
        f = x[part].cpu().double()
        ref.check(mean[part], wm, f.abs().mean(-1), K, "mean")
        size = (f.abs() + f.abs().mean(-1, keepdim=True)) * wr[..., None]
        ref.check(y[part], wy, 2 * size * 1.5 + 0.5, K, "y")
        want, mag = ref.layer_norm_backward(dy[part], x[part], mean[part], rstd[part], weight)
        ref.check(dx[part], want[0], 2 * mag[0], K, "dx")
    total = torch.zeros(C, dtype=torch.float64)
    size = torch.zeros(C, dtype=torch.float64)
    for i in range(0, rows, 1_000_000):
        total += dy[i:i + 1_000_000].double().sum(0).cpu()
        size += dy[i:i + 1_000_000].double().abs().sum(0).cpu()
    # a slab adds rows / 1024 / 16 of them one by one in a lane, then lanes and slabs
    ref.check(db, total, size, rows / 1024 / 16 + 16 + 1024, "dbias")


def test_longest_row():
    # 2^31 - 1 values of +1 and -1 in turn: every sum is exact, mean 2^-31, variance 1
    C = (1 << 31) - 1
    print(f"[case] one row of {C}", flush=True)
    x = torch.ones(C, device="cuda", dtype=torch.bfloat16)
    x[1::2] = -1
    y, mean, rstd = gdn.layer_norm(x.view(1, C), stats=True)
    dx, dw, db = gdn.layer_norm_backward(x.view(1, C), x.view(1, C), mean, rstd, params=True)
    torch.cuda.synchronize()
    assert abs(float(mean) * C - 1) < 1e-6 and abs(float(rstd) - 1 / math.sqrt(1 + 1e-5)) < 1e-6
    assert torch.equal(y[0], x) and torch.equal(db.bfloat16(), x)
    # r (g - sum(g) / C - n sum(g n) / C) = r (1 - r^2) x = 1e-5 x, to a few roundings of 1
    assert float(dx.abs().max()) < 1.2e-5
    assert float((dw - rstd).abs().max()) < 1e-6
