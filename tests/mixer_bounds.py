"""The gated Mamba-1 scan and its gradient in 64 bits on the CPU, with a bound on what a
float32 evaluation can be off by, element by element.

mixer_ref multiplies one count of roundings for a whole sequence with the sum of
magnitudes.  Here the error of each state is carried along with it and decays as it does,
so that the bound does not grow with the length of a sequence whose states forget.  Errors
are in units of 2^-24; first order (the squares are below 2^-40).

``seg``: the tokens of a segment where the sequence is cut (its carried decay is the
exponential of a sum of up to that many steps, each addition rounded), 0 where it is not.
"""
import torch

from mixer_ref import U32, dsilu, silu, spans, step_size


def within(got, want, what=""):
    """|got - ref| <= half a step of got's type + 2^-24 error."""
    ref, err = want
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + U32 * err + 1e-30
    if got.dtype == torch.bfloat16:  # the rounding acts on the float32 value
        tol = tol * (1 + 2.0 ** -7)
    bad = (g - ref).abs() > tol
    assert torch.isfinite(g).all() and not bad.any(), (
        f"{what}: {int(bad.sum())} of {g.numel()} off, worst {float(((g - ref).abs() / tol).max()):.2f} of the tolerance")


class Scan:
    """The forward's values and errors, kept token by token for the gradient."""

    def __init__(self, x, dt, A, B, C, cu, D=None, z=None, bias=None, softplus=True, init=None, seg=0):
        self.ins, self.cu, self.D, self.z, self.softplus = (x, A, B, C), cu, D, z, softplus
        n, d = x.shape
        N, G = A.shape[1], B.shape[1]
        self.of = of = torch.arange(d) // (d // G)
        self.raw, self.delta = raw, delta = step_size(dt, bias, softplus)
        # softplus: its argument is rounded, scaled and rounded (3 |v| in the exponent), the
        # exponential is good to 2^-22; the quotient, the series and the last sum make 12
        self.kd = kd = 4 * raw.abs() + 16 if softplus else torch.ones_like(raw)
        self.kz = None if z is None else 3 * z.abs() + 10  # the gate: the same, a reciprocal and a product
        zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
        self.y, self.ey = zero(n, d), zero(n, d)
        nseq = cu.numel() - 1
        self.end, self.eend = zero(nseq, d, N), zero(nseq, d, N)
        self.h, self.m, self.eh = [None] * n, [None] * n, [None] * n  # after each token
        self.p, self.mp, self.ep = zero(n, d), zero(n, d), zero(n, d)  # before the gate
        for i, (lo, hi) in enumerate(spans(cu)):
            h = zero(d, N) if init is None else init[i].clone()
            m, e = h.abs(), zero(d, N)
            for t in range(lo, hi):
                a, ka = self.decay(t, seg)
                b = (delta[t] * x[t])[:, None] * B[t][of]
                e = a * (e + ka * m) + (kd[t][:, None] + 3) * b.abs()
                h, m = a * h + b, a * m + b.abs()
                e = e + m
                self.h[t], self.m[t], self.eh[t] = h, m, e
                c = C[t][of]
                skip = torch.zeros(d, dtype=torch.float64) if D is None else D * x[t]
                p = (h * c).sum(1) + skip
                mp = (m * c.abs()).sum(1) + skip.abs()
                ep = (e * c.abs()).sum(1) + (N + 6) * mp
                self.p[t], self.mp[t], self.ep[t] = p, mp, ep
                gate = 1.0 if z is None else silu(z[t])
                self.y[t] = p * gate
                self.ey[t] = ep if z is None else (ep + (self.kz[t] + 1) * mp) * gate.abs()
            self.end[i], self.eend[i] = h, e
        self.seg = seg

    def decay(self, t, seg):
        """exp(delta A) and its relative error: that of its argument, and 2^-22."""
        arg = self.delta[t][:, None] * self.ins[1]
        return torch.exp(arg), arg.abs() * (self.kd[t][:, None] + 3 + seg) + 4

    def bwd(self, dy):
        """dict of (gradient, error)."""
        x, A, B, C = self.ins
        (n, d), (N, G), of, delta, kd = x.shape, (A.shape[1], B.shape[1]), self.of, self.delta, self.kd
        gate = 1.0 if self.z is None else silu(self.z)
        dp = dy * gate
        kdp = torch.ones_like(dy) if self.z is None else self.kz + 1
        zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
        names = dict(dx=(n, d), ddt=(n, d), dA=(d, N), dB=(n, G, N), dC=(n, G, N), dD=(d,), dz=(n, d), ddt_bias=(d,))
        g, E = {k: zero(*s) for k, s in names.items()}, {k: zero(*s) for k, s in names.items()}
        Dv = zero(d) if self.D is None else self.D
        group = lambda v: v.unflatten(0, (G, d // G)).sum(1)  # noqa: E731
        chan = 2 * (d // G) + 8  # a sum over channels: products kept to 2^-22, each addition within a step
        for lo, hi in spans(self.cu):
            acc = (hi - lo) // 4 + 8  # additions of a long sum over tokens, four at a time
            carry, mc, ec = zero(d, N), zero(d, N), zero(d, N)
            for t in range(hi - 1, lo - 1, -1):
                a, ka = self.decay(t, self.seg)
                c, b, kdt = C[t][of], B[t][of], kd[t][:, None]
                own = dp[t][:, None] * c
                gh, mh = own + carry, own.abs() + mc
                eg = own.abs() * (kdp[t][:, None] + 1) + ec + mh
                h, m, eh = (self.h[t - 1], self.m[t - 1], self.eh[t - 1]) if t > lo else (zero(d, N),) * 3
                carry, mc, ec = a * gh, a * mh, a * (eg + (ka + 1) * mh)
                q, mq = carry * h, mc * m
                eq = ec * m + mc * eh + mq
                du, mu = (gh * b).sum(1), (mh * b.abs()).sum(1)
                edu = (eg * b.abs()).sum(1) + (N + 6) * mu
                g["dx"][t] = delta[t] * du + Dv * dp[t]
                E["dx"][t] = delta[t].abs() * (edu + (kd[t] + 2) * mu) + (Dv * dp[t]).abs() * (kdp[t] + 2)
                raw = self.raw[t]
                sg = torch.sigmoid(raw) if self.softplus else torch.ones_like(raw)
                md = x[t].abs() * mu + (mq * A.abs()).sum(1)
                g["ddt"][t] = (x[t] * du + (q * A).sum(1)) * sg
                E["ddt"][t] = (x[t].abs() * edu + (eq * A.abs()).sum(1) + (N + 10) * md
                               + (3 * raw.abs() + 10 if self.softplus else 1) * md) * sg
                g["ddt_bias"] += g["ddt"][t]
                E["ddt_bias"] += E["ddt"][t] + acc * md * sg
                g["dA"] += delta[t][:, None] * q
                E["dA"] += delta[t].abs()[:, None] * (eq + (kdt + 3 + acc) * mq)
                u = (delta[t] * x[t])[:, None]
                g["dB"][t] = group(u * gh)
                E["dB"][t] = group(u.abs() * (eg + (kdt + 2 + chan) * mh))
                g["dC"][t] = group(dp[t][:, None] * self.h[t])
                E["dC"][t] = group(dp[t].abs()[:, None] * (self.eh[t] + (kdp[t][:, None] + 2 + chan) * self.m[t]))
                g["dD"] += dp[t] * x[t]
                E["dD"] += (dp[t] * x[t]).abs() * (kdp[t] + 2 + acc * 4)
                if self.z is not None:
                    z, s = self.z[t], torch.sigmoid(self.z[t])
                    g["dz"][t] = dy[t] * self.p[t] * dsilu(z)
                    # silu' by its two terms, each with the gate's error
                    E["dz"][t] = dy[t].abs() * (dsilu(z).abs() * (self.ep[t] + 4 * self.mp[t])
                                                + self.p[t].abs() * s * (1 + z.abs()) * (self.kz[t] + 6))
        return {k: (g[k], E[k]) for k in g}
