"""64-bit references of the rotation and the norm of queries and keys, and the bars of their tests.

A result in a type T is off by at most half a step (finfo(T).eps / 2 relative) from its rounding, and by the
fp32 arithmetic before it. In units of u = 2^-24 (half a step of 1 in fp32):
  the angle, reduced in 64 bits, is rounded once as half turns of at most 1: pi u / 2 < 2 u radians; cosine and
  sine are then off by that and 4 steps (8 u) of their own; two products and a sum add 3 u of |x| + |y|: a
  rotation is off by at most 16 u amplitude (|x| + |y|), taken as 32 u = 2^-19.
  the norm: the sum of squares adds up to 16 terms in a lane and 6 levels of lanes (22 u), the mean, the root, the
  quotient and the products with r and w a step or two each: (22 / 2 + 10) u, taken with the rotation's as 64 u = 2^-18.
  its gradient forms another such sum and subtracts: 128 u = 2^-17 of the terms' magnitudes.
  the weights' gradient sums N rows of that: at most min(N, 2048) + 300 additions in a row (a lane's share, the lanes
  and waves of a workgroup, the slabs, the heads), one u each."""
import torch

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(ref, dtype):
    """Half a step of `dtype` at ref, and half the smallest subnormal."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def angles(positions, freqs, B, T):
    """[B, T, 1, R/2] angles in 64 bits."""
    p = torch.arange(T).expand(B, T) if positions is None else positions
    return (p.double()[..., None] * freqs)[:, :, None]


def rotate(x, theta, amplitude, interleaved, transposed=False):
    """x [B, T, H, D] in 64 bits, R = 2 * theta.shape[-1]."""
    r = theta.shape[-1]
    c, s = torch.cos(theta) * amplitude, torch.sin(theta) * amplitude
    if transposed:
        s = -s
    rot, rest = x[..., :2 * r], x[..., 2 * r:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        out = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = rot[..., :r], rot[..., r:]
        out = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([out, rest], -1)


def reach(x, theta, amplitude, interleaved):
    """amplitude (|x| + |y|) at both members of each pair, |x| past them: what the rotation's errors scale with."""
    r = theta.shape[-1]
    rot, rest = x[..., :2 * r].abs(), x[..., 2 * r:].abs()
    if interleaved:
        both = (rot[..., 0::2] + rot[..., 1::2]) * abs(amplitude)
        out = torch.stack([both, both], -1).flatten(-2)
    else:
        both = (rot[..., :r] + rot[..., r:]) * abs(amplitude)
        out = torch.cat([both, both], -1)
    return torch.cat([out, rest], -1)


def cut(x, lengths):
    """Rows past the lengths as zeros."""
    if lengths is None:
        return x
    t = torch.arange(x.shape[1])
    keep = t[None, :] < lengths.clamp(0, x.shape[1])[:, None]
    return torch.where(keep[:, :, None, None], x, torch.zeros_like(x))


def norm(x, w, eps):
    """(x r w, r) in 64 bits."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x * r
    return (y if w is None else y * w), r


def norm_grads(x, dy, w, eps, theta, amplitude, interleaved, lengths):
    """dx, dw [H, D] and their bars (before the rounding of the result), in 64 bits from the formulas."""
    x, dy = cut(x, lengths), cut(dy, lengths)
    one = torch.ones((), dtype=torch.float64) if w is None else w
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    g = rotate(dy, theta, amplitude, interleaved, transposed=True)
    G = reach(dy, theta, amplitude, interleaved)
    t = g * one
    dx = cut(r * (t - n * (t * n).mean(-1, keepdim=True)), lengths)
    size = r * (G * one.abs() + n.abs() * (G * one.abs() * n.abs()).mean(-1, keepdim=True))
    N = x.shape[0] * x.shape[1]
    dw = (g * n).sum((0, 1))
    dw_size = (G * n.abs()).sum((0, 1))
    return dx, dw, cut(size, lengths) * 128 * U, dw_size * U * (64 + min(N, 2048) + 300)
