"""A 64-bit reference of the gated linear recurrence, token by token, and the bars of its tests.

In units of u = 2^-24 (half a step of 1 in fp32) the kernels' gates are off by: e^-|a| 4 u; sigmoids (a sum, a
reciprocal of 2 u, a product) 8 u; softplus (1 + w, a logarithm of 2 u) 8 u; 1 - alpha, from its series or by
difference, 32 u of itself; alpha, where it stands for itself (below 1/2), less than 32 u (1 - alpha). So a token adds to
the error of h: 32 u (1 - alpha) |h|, 16 u of beta |x|, and 8 u of the magnitude for the operations themselves (the map's
product and sum, its composition and the state's update). The bars carry these sums along the sequence as the
recurrence carries h: E <- alpha E + u (32 (1 - alpha) A + 16 beta |x| + 8 A), with A the recurrence of |x|. The
adjoint g has the same bar backwards. A result is rounded once more to its own type (half a step).
The exponential instruction returns 0 for results below 2^-126, the smallest normal number: an alpha, and e^-|a| with the
sigmoids made of it, may be off by that much outright (alpha = e^-88 counts as 0), which what multiplies them scales."""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 64


def half_step(ref, dtype):
    """Half a step of `dtype` at ref, and half the smallest subnormal."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def gates(a, b, rate):
    """alpha, 1 - alpha, beta, softplus(a) in 64 bits; rate [C] or None, b None: beta = 1 - alpha."""
    soft = torch.logaddexp(a, torch.zeros_like(a))
    e = soft if rate is None else soft * rate
    alpha, lost = torch.exp(-e), -torch.expm1(-e)
    return alpha, lost, lost if b is None else torch.sigmoid(b), soft


class Forward:
    """States h, their bars E and magnitudes A [B, T + 1, C] (before the first token and after each), from
    64-bit inputs; the tokens past the lengths change nothing."""

    def __init__(self, x, a, b, rate, state, lengths):
        B, T, C = x.shape
        self.alpha, self.lost, self.beta, self.soft = gates(a, b, rate)
        n = torch.full((B,), T) if lengths is None else lengths.clamp(0, T)
        self.here = (torch.arange(T)[None, :] < n[:, None])[..., None]
        h = torch.zeros(B, C, dtype=torch.float64) if state is None else state
        A, E = h.abs(), torch.zeros_like(h)
        hs, As, Es = [h], [A], [E]
        for t in range(T):
            al, lo, be, on = self.alpha[:, t], self.lost[:, t].abs(), self.beta[:, t], self.here[:, t]
            # (no state, a zero state or x may be infinite elsewhere: tokens that are not there are not computed)
            xt = torch.where(on, x[:, t], torch.zeros_like(h))
            h = torch.where(on, al * h + be * xt, h)
            E = torch.where(on, al * E + U * (32 * lo * A + 16 * (be * xt).abs() + 8 * (A + (be * xt).abs())) + TINY * (A + xt.abs()), E)
            A = torch.where(on, al * A + (be * xt).abs(), A)
            hs.append(h), As.append(A), Es.append(E)
        self.h, self.A, self.E = (torch.stack(z, 1) for z in (hs, As, Es))

    def outputs(self):
        """o [B, T, C] and its bar, zeros past the lengths."""
        zero = torch.zeros_like(self.h[:, 1:])
        return torch.where(self.here, self.h[:, 1:], zero), torch.where(self.here, self.E[:, 1:], zero)

    def kept(self):
        """The states before the tokens 0, 64, ... and their bars."""
        return self.h[:, :-1:CHUNK], self.E[:, :-1:CHUNK]


def backward(f, x, a, b, rate, d_o, dstate):
    """{name: (gradient, bar)} from the formulas."""
    B, T, C = x.shape
    zero = torch.zeros(B, C, dtype=torch.float64)
    g = zero if dstate is None else dstate
    G, E = g.abs(), zero
    out = {n: [None] * T for n in ("dx", "da", "db", "e")}
    r = torch.ones(C, dtype=torch.float64) if rate is None else rate
    for t in range(T - 1, -1, -1):
        al, lo, be, on = f.alpha[:, t], f.lost[:, t].abs(), f.beta[:, t], f.here[:, t]
        sl = torch.sigmoid(a[:, t]) * r
        d = torch.where(on, d_o[:, t], zero)
        xt = torch.where(on, x[:, t], zero)
        now, mag, err = g + d, G + d.abs(), E + U * (G + d.abs())
        before, Ab, Eb = f.h[:, t], f.A[:, t], f.E[:, t]
        e = now * al * ((xt if b is None else 0) - before)
        size = Ab + (xt.abs() if b is None else 0)
        da_err = al * (err * size + mag * Eb + 80 * U * mag * size) + TINY * mag * size
        keep = lambda v: torch.where(on, v, zero)  # noqa: E731
        out["dx"][t] = (keep(now * be), keep(be.abs() * (err + 40 * U * mag) + TINY * mag))
        out["e"][t] = (keep(e), keep(da_err))
        out["da"][t] = (keep(e * sl), keep(sl.abs() * (da_err + 16 * U * al * mag * size) + TINY * r.abs() * al * mag * size))
        if b is not None:
            s = be * torch.sigmoid(-b[:, t])
            out["db"][t] = (keep(now * xt * s), keep(s * xt.abs() * (err + 40 * U * mag) + TINY * mag * xt.abs()))
        g = torch.where(on, al * now, g)
        E = torch.where(on, al * err + U * (32 * lo * mag + 8 * mag) + TINY * mag, E)
        G = torch.where(on, al * mag, G)
    res = {n: tuple(torch.stack([p[i] for p in out[n]], 1) for i in (0, 1)) for n in out if out[n] and out[n][0] is not None}
    if T:
        e, err = res.pop("e")
        soft = torch.where(f.here, f.soft, torch.zeros_like(f.soft))
        # a chunk's 64 terms in 32 bits, the chunks in 64
        res["drate"] = ((e * soft).sum((0, 1)), (soft * (err + 80 * U * e.abs())).sum((0, 1)))
    res["dstate0"] = (g, E)
    return res
