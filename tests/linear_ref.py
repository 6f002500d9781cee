"""64-bit references and error bounds for linear attention with a decay for each head and for layer
norm (used by the gpu-marked tests of both).

The references follow the definitions token by token in fp64. Beside each result they give its
magnitude: the same sums with every term's absolute value. Bounds count roundings against it:
  * an fp32 result is a sum whose terms each pass through at most K roundings of 2^-24 relative, so
    |x - ref| <= K 2^-24 mag elementwise (Higham's bound, to first order). Roundings are not all
    alike, so the error's 2-norm stays near that of a random walk: ||x - ref|| <= 2 sqrt(K) 2^-24 ||mag||.
    Attention: K = 2 T + D + 16 (two per token of the recurrence, D of a product, the factors);
    layer norm over C: K = C / 64 + 32 (a lane's own terms, then a tree; the factors).
  * 16-bit outputs of attention may hold the fp32 state and the weighted scores as two bf16 parts
    (at most 2^-16 of a term is lost in each, and in the dropped product of the low parts): 2^-14 mag
    more covers them. That slack does not apply to fp32 outputs.
  * rounding to a 16-bit type adds half a step: eps / 2 of the value, or half the smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

HALF = {torch.float32: 0.0, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float16: torch.finfo(torch.float16).eps / 2}
SUB = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
U = 2.0 ** -24


def _f(t):
    return None if t is None else t.detach().cpu().double()


def _heads(x, H):
    return x.repeat_interleave(H // x.shape[2], dim=2)


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths.cpu()]


def forward(q, k, v, decay, state, scale, lengths=None):
    """(o, state after) in fp64."""
    q, k, v, decay, S = _f(q), _f(k), _f(v), _f(decay), _f(state).clone()
    B, T, H, D = v.shape
    q, k = _heads(q, H), _heads(k, H)
    o = torch.zeros_like(v)
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            S[b] = decay[:, None, None] * S[b] + v[b, t][:, :, None] * k[b, t][:, None, :]
            o[b, t] = scale * (S[b] * q[b, t][:, None, :]).sum(-1)
    return o, S


def forward_mag(q, k, v, decay, state, scale, lengths=None):
    return forward(q.abs(), k.abs(), v.abs(), decay.abs(), state.abs(), abs(scale), lengths)


def backward(q, k, v, decay, d_o, state0, dstate, scale, lengths=None):
    """(dq, dk, dv, dstate0, ddecay) in fp64, from the adjoint recurrence."""
    Hk = q.shape[2]
    q, k, v, decay, d_o = _f(q), _f(k), _f(v), _f(decay), _f(d_o)
    B, T, H, D = v.shape
    q, k = _heads(q, H), _heads(k, H)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(v)
    dS0 = torch.zeros(B, H, D, D, dtype=torch.float64)
    dl = torch.zeros(H, dtype=torch.float64)
    lam = decay[:, None, None]
    for b, n in enumerate(_lengths(lengths, B, T)):
        S = [torch.zeros(H, D, D, dtype=torch.float64) if state0 is None else _f(state0)[b]]
        for t in range(n):
            S.append(lam * S[-1] + v[b, t][:, :, None] * k[b, t][:, None, :])
        R = torch.zeros(H, D, D, dtype=torch.float64) if dstate is None else _f(dstate)[b]
        for t in reversed(range(n)):
            R = R + scale * d_o[b, t][:, :, None] * q[b, t][:, None, :]
            dq[b, t] = scale * (S[t + 1] * d_o[b, t][:, :, None]).sum(1)
            dk[b, t] = (R * v[b, t][:, :, None]).sum(1)
            dv[b, t] = (R * k[b, t][:, None, :]).sum(2)
            dl += (R * S[t]).sum((1, 2))
            R = lam * R
        dS0[b] = R
    fold = lambda x: x.reshape(B, T, Hk, H // Hk, D).sum(3)  # noqa: E731
    return fold(dq), fold(dk), dv, dS0, dl


def backward_mag(q, k, v, decay, d_o, state0, dstate, scale, lengths=None):
    a = lambda x: None if x is None else x.abs()  # noqa: E731
    return backward(q.abs(), k.abs(), v.abs(), decay.abs(), d_o.abs(), a(state0), a(dstate), abs(scale), lengths)


def attn_roundings(T, D):
    return 2 * T + D + 16


def check(got, ref, mag, K, what, parts=False):
    """Holds `got` (a tensor of its own type) to the bounds above."""
    dt = got.dtype
    got = _f(got)
    ref, mag = torch.as_tensor(ref), torch.as_tensor(mag)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    slack = 2.0 ** -14 if parts and dt != torch.float32 else 0.0
    err = (got - ref).abs()
    bound = (K * U + slack) * mag * (1 + HALF[dt]) + HALF[dt] * ref.abs() + SUB[dt] + 1e-40
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its elementwise bound"
    if dt == torch.float32 and err.numel():
        r, m = float(err.norm()), float(mag.norm())
        assert r <= 2 * np.sqrt(K) * U * m + 1e-40, f"{what}: 2-norm error {r / max(m, 1e-300):.3g} of the magnitude"
    return worst


def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd) in fp64; weight and bias [C] or [G, C] or None."""
    x = _f(x)
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mean) * rstd
    y = y * (1 if weight is None else _f(weight)) + (0 if bias is None else _f(bias))
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_backward(dy, x, mean, rstd, weight):
    """(dx, dw, db) and their magnitudes, in fp64, with the given statistics; dw, db summed over
    all but weight's dimensions (the last one without weight)."""
    dy, x, m, r = _f(dy), _f(x), _f(mean)[..., None], _f(rstd)[..., None]
    n = (x - m) * r
    nm = (x.abs() + m.abs()) * r
    w = torch.ones((), dtype=torch.float64) if weight is None else _f(weight)
    g = dy * w
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    ga = g.abs()
    dxm = r * (ga + ga.mean(-1, keepdim=True) + nm * (ga * nm).mean(-1, keepdim=True))
    keep = weight.dim() if weight is not None else 1
    dims = tuple(range(x.dim() - keep))
    red = (lambda t: t.sum(dims)) if dims else (lambda t: t)
    return (dx, red(dy * n), red(dy)), (dxm, red(dy.abs() * nm), red(dy.abs()))
