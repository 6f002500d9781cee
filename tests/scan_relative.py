"""Bars of the gated linear recurrence that scale with what is left of a state, not with the state before a token: a token
that forgets keeps alpha h and beta x to fp32's own steps, however large h was. The references are scan_ref.py's.

In units of u = 2^-24. alpha = e^-s with s = rate softplus(a): softplus is off by 8 u, the product by 1 u, so alpha by
9 s u, the exponential by 2 u and, where it is formed from 1 - alpha (s < 1/8), by 32 s u in all. Of 16-bit gates the
exponent a log2 e is rounded too, |a| u of the result where that is alpha itself (a > 0 without a rate, where |a| < s) and |a| u of
softplus elsewhere, |a| s u of alpha. So W = s (32 + |a|) + 8 bounds alpha's relative error in u. beta = sigmoid(b) is off
by 16 u (scan_ref.py), beta = 1 - alpha by 32 u from its series and by alpha W / |1 - alpha| by difference; and the map's product and sum, its
composition and the state's update each round the result, 8 u of the new magnitude alpha A + beta |x| in all. So

    E <- alpha E + u (alpha A W + WB beta |x| + 8 (alpha A + beta |x|)) + 2^-126 (A + |x|)

(+ SUB: a product or sum below 2^-126 is a multiple of 2^-149, off by up to 2^-150 whatever its size; a token's map has two, and
so have the two-step products of da and db, g (x - h) times sigmoid(a) rate and g x times beta (1 - beta), before their last
rounding: with g, x and h of 1e-30 the first product, 1e-60, has no relative bar at all), with WB = 16, or 40 + alpha W / |1 - alpha| (s >= 1/10) without b. The adjoint has the same bar backwards."""
import torch

from scan_ref import TINY, U, Forward

SUB = 2.0 ** -149


class Relative(Forward):
    """Forward with these bars in place of its own."""

    def __init__(self, x, a, b, rate, state, lengths):
        super().__init__(x, a, b, rate, state, lengths)
        s = (self.soft if rate is None else self.soft * rate).abs()
        finite = torch.where(a.isfinite(), a.abs(), torch.zeros_like(a))
        self.W = torch.where(self.alpha == 0, torch.zeros_like(s), s * (32 + finite) + 8)
        self.WB = torch.full_like(s, 16)
        if b is None:
            by_difference = self.alpha * self.W / self.lost.abs().clamp(min=0.05)
            self.WB = 40 + torch.where(s > 0.1, by_difference, torch.zeros_like(s))
        E = torch.zeros_like(self.h[:, 0])
        Es = [E]
        for t in range(x.shape[1]):
            al, A, on = self.alpha[:, t], self.A[:, t], self.here[:, t]
            xt = torch.where(on, x[:, t], torch.zeros_like(A))
            u = (self.beta[:, t] * xt).abs()
            step = al * E + U * (al * A * self.W[:, t] + self.WB[:, t] * u + 8 * (al * A + u)) + TINY * (A + xt.abs()) + SUB
            E = torch.where(on, step, E)
            Es.append(E)
        self.E = torch.stack(Es, 1)


def backward(f, x, a, b, rate, d_o, dstate):
    """{name: (gradient, bar)} from the formulas, f a Relative."""
    B, T, C = x.shape
    zero = torch.zeros(B, C, dtype=torch.float64)
    g = zero if dstate is None else dstate
    G, E = g.abs(), zero
    out = {n: [None] * T for n in ("dx", "da", "e", *(() if b is None else ("db",)))}
    r = torch.ones(C, dtype=torch.float64) if rate is None else rate
    for t in range(T - 1, -1, -1):
        al, be, W, on = f.alpha[:, t], f.beta[:, t], f.W[:, t], f.here[:, t]
        sl = torch.sigmoid(a[:, t]) * r
        d = torch.where(on, d_o[:, t], zero)
        xt = torch.where(on, x[:, t], zero)
        now, mag, err = g + d, G + d.abs(), E + U * (G + d.abs())
        size = f.A[:, t] + (xt.abs() if b is None else 0)
        e = now * al * ((xt if b is None else 0) - f.h[:, t])
        e_err = al * (err * size + mag * f.E[:, t] + (W + 24) * U * mag * size) + TINY * mag * size + SUB

        def keep(v):
            return torch.where(on, v, zero)
        out["dx"][t] = (keep(now * be), keep(be.abs() * (err + (f.WB[:, t] + 8) * U * mag) + TINY * mag))
        out["e"][t] = (keep(e), keep(e_err))
        out["da"][t] = (keep(e * sl), keep(sl.abs() * (e_err + 24 * U * al * mag * size) + TINY * r.abs() * al * mag * size))
        if b is not None:
            s = be * torch.sigmoid(-b[:, t])
            out["db"][t] = (keep(now * xt * s), keep(s * xt.abs() * (err + 40 * U * mag) + TINY * mag * xt.abs() + SUB))
        g = torch.where(on, al * now, g)
        E = torch.where(on, al * err + U * al * mag * (W + 8) + TINY * mag + SUB, E)
        G = torch.where(on, al * mag, G)
    res = {n: tuple(torch.stack([p[i] for p in out[n]], 1) for i in (0, 1)) for n in out}
    e, err = res.pop("e")
    soft = torch.where(f.here, f.soft, torch.zeros_like(f.soft))
    # a chunk's 64 terms in 32 bits, the chunks in 64
    res["drate"] = ((e * soft).sum((0, 1)), (soft * (err + 80 * U * e.abs())).sum((0, 1)))
    res["dstate0"] = (g, E)
    return res
