"""The mixer-block operators in 64 bits, straight from their formulas, on the CPU.

Each function also gives the magnitude M of what it sums: the same formula with
every product taken absolutely.  A float32 evaluation that rounds k times on the
way to an output is off by at most about k 2^-24 M, and storing it in the io type
adds half a step of the value itself; ``close`` checks that, element by element.
"""
import torch

U32 = 2.0 ** -24


def close(got, ref, mag, roundings, what="", fits=None):
    """|got - ref| <= half a step of got's type + roundings * 2^-24 * mag, where fits."""
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    if fits is not None:
        g, ref, mag = g[fits], ref[fits], mag[fits]
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + roundings * U32 * mag + 1e-30
    if got.dtype == torch.bfloat16:  # the rounding acts on the float32 value, itself off by the second term
        tol = tol * (1 + 2.0 ** -7)
    bad = (g - ref).abs() > tol
    assert torch.isfinite(g).all() and not bad.any(), (
        f"{what}: {int(bad.sum())} of {g.numel()} off, worst {float(((g - ref).abs() / tol).max()):.2f} of the tolerance")


def d64(t):
    return None if t is None else t.detach().double().cpu()


def silu(v):
    return v * torch.sigmoid(v)


def dsilu(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def spans(cu):
    cu = cu.tolist()
    return [(cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


# ------------------------------------------------------------------ convolution

def conv(x, w, b, cu, act, init=None):
    """(out, magnitude, last inputs [nseq, C, K-1]); init [nseq, C, K-1] or None.
    Rows of no sequence stay zero."""
    n, c = x.shape
    K = w.shape[1]
    out, mag = torch.zeros(n, c, dtype=torch.float64), torch.zeros(n, c, dtype=torch.float64)
    last = torch.zeros(cu.numel() - 1, c, K - 1, dtype=torch.float64)
    for i, (lo, hi) in enumerate(spans(cu)):
        old = torch.zeros(K - 1, c, dtype=torch.float64) if init is None else init[i].T
        seq = torch.cat([old, x[lo:hi]])
        last[i] = seq[seq.shape[0] - (K - 1):].T
        for t in range(hi - lo):
            win = seq[t:t + K]
            pre = (win * w.T).sum(0) + (0 if b is None else b)
            am = (win * w.T).abs().sum(0) + (0 if b is None else b.abs())
            out[lo + t] = silu(pre) if act else pre
            mag[lo + t] = am * 1.1 if act else am  # |silu'| < 1.1
    return out, mag, last


def conv_bwd(x, w, b, cu, dout, act):
    """dict of (gradient, magnitude) for dxbc, dweight, dbias."""
    n, c = x.shape
    K = w.shape[1]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    dx, mx, dw, mw, db, mb = z(n, c), z(n, c), z(c, K), z(c, K), z(c), z(c)
    for lo, hi in spans(cu):
        seq = torch.cat([z(K - 1, c), x[lo:hi]])
        for t in range(hi - lo):
            win = seq[t:t + K]
            pre = (win * w.T).sum(0) + (0 if b is None else b)
            am = (win * w.T).abs().sum(0) + (0 if b is None else b.abs())
            d = dout[lo + t] * (dsilu(pre) if act else 1.0)
            md = dout[lo + t].abs() * (1.1 + 0.5 * am if act else 1.0)  # |silu''| <= 1/2 carries the error of pre
            for j in range(min(K, t + 1)):
                dx[lo + t - j] += w[:, K - 1 - j] * d
                mx[lo + t - j] += w[:, K - 1 - j].abs() * md
            dw += (win * d).T
            mw += (win.abs() * md).T
            db += d
            mb += md
    return dict(dxbc=(dx, mx), dweight=(dw, mw), dbias=(db, mb))


# --------------------------------------------------------------- selective scan

def step_size(dt, bias, softplus):
    raw = dt if bias is None else dt + bias
    return raw, (torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())) if softplus else raw)


def sel(x, dt, A, B, C, cu, D=None, z=None, bias=None, softplus=True, init=None):
    """(y, magnitude, end states [nseq, d, N], their magnitude, states before every 128th token by sequence)."""
    n, d = x.shape
    N, G = A.shape[1], B.shape[1]
    of = torch.arange(d) // (d // G)
    _, delta = step_size(dt, bias, softplus)
    y, my = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    ends, mends, kept = [], [], []
    for i, (lo, hi) in enumerate(spans(cu)):
        h = torch.zeros(d, N, dtype=torch.float64) if init is None else init[i].clone()
        m, states = h.abs(), []
        for t in range(lo, hi):
            if (t - lo) % 128 == 0:
                states.append(h)
            a = torch.exp(delta[t][:, None] * A)
            b = (delta[t] * x[t])[:, None] * B[t][of]
            h, m = a * h + b, a * m + b.abs()
            y[t] = (h * C[t][of]).sum(1) + (0 if D is None else D * x[t])
            my[t] = (m * C[t][of].abs()).sum(1) + (0 if D is None else (D * x[t]).abs())
            if z is not None:
                y[t] *= silu(z[t])
                my[t] *= silu(z[t]).abs()
        ends.append(h)
        mends.append(m)
        kept.append(states)
    return y, my, torch.stack(ends), torch.stack(mends), kept


def growth_fits(dt, A, cu, bias=None, softplus=True):
    """[nseq, d]: whether no product of a sequence's decays leaves float32 (2^128).  Only
    steps below zero grow; the scan forms exp(A sum of delta) over up to 512 tokens, so
    past that bound its factors are infinite even where the state they multiply is not."""
    _, delta = step_size(dt, bias, softplus)
    total = [torch.clamp(delta[lo:hi, :, None] * A, min=0).sum(0).amax(1) for lo, hi in spans(cu)]
    return torch.stack(total) * 1.4427 < 126


def sel_bwd(x, dt, A, B, C, cu, dy, D=None, z=None, bias=None, softplus=True):
    """dict of (gradient, magnitude)."""
    n, d = x.shape
    N, G = A.shape[1], B.shape[1]
    of = torch.arange(d) // (d // G)
    raw, delta = step_size(dt, bias, softplus)
    gate = 1.0 if z is None else silu(z)
    dyp = dy * gate
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    names = dict(dx=(n, d), ddt=(n, d), dA=(d, N), dB=(n, G, N), dC=(n, G, N), dD=(d,), dz=(n, d), ddt_bias=(d,))
    g = {k: zero(*s) for k, s in names.items()}
    M = {k: zero(*s) for k, s in names.items()}
    Dv = zero(d) if D is None else D
    group = lambda v: v.unflatten(0, (G, d // G)).sum(1)  # noqa: E731
    for lo, hi in spans(cu):
        h, m = [zero(d, N)], [zero(d, N)]
        for t in range(lo, hi):
            a = torch.exp(delta[t][:, None] * A)
            b = (delta[t] * x[t])[:, None] * B[t][of]
            h.append(a * h[-1] + b)
            m.append(a * m[-1] + b.abs())
            if z is not None:
                pre = (h[-1] * C[t][of]).sum(1) + Dv * x[t]
                mp = (m[-1] * C[t][of].abs()).sum(1) + (Dv * x[t]).abs()
                g["dz"][t] = dy[t] * pre * dsilu(z[t])
                M["dz"][t] = (dy[t] * dsilu(z[t])).abs() * mp + (dy[t] * pre).abs()  # silu' itself: a few roundings of 1
        carry, mc = zero(d, N), zero(d, N)
        for t in range(hi - 1, lo - 1, -1):
            a = torch.exp(delta[t][:, None] * A)
            gh = dyp[t][:, None] * C[t][of] + carry
            mh = (dyp[t][:, None] * C[t][of]).abs() + mc
            before, mb = h[t - lo], m[t - lo]
            q, mq = gh * a * before, mh * a * mb
            du, mu = (gh * B[t][of]).sum(1), (mh * B[t][of].abs()).sum(1)
            g["dx"][t] = delta[t] * du + Dv * dyp[t]
            M["dx"][t] = delta[t].abs() * mu + (Dv * dyp[t]).abs()
            sg = torch.sigmoid(raw[t]) if softplus else 1.0
            g["ddt"][t] = (x[t] * du + (q * A).sum(1)) * sg
            M["ddt"][t] = (x[t].abs() * mu + (mq * A.abs()).sum(1)) * sg
            g["dA"] += delta[t][:, None] * q
            M["dA"] += delta[t].abs()[:, None] * mq
            g["dB"][t] = group((delta[t] * x[t])[:, None] * gh)
            M["dB"][t] = group((delta[t] * x[t]).abs()[:, None] * mh)
            g["dC"][t] = group(dyp[t][:, None] * h[t - lo + 1])
            M["dC"][t] = group(dyp[t].abs()[:, None] * m[t - lo + 1])
            g["dD"] += dyp[t] * x[t]
            M["dD"] += (dyp[t] * x[t]).abs()
            carry, mc = a * gh, a * mh
    g["ddt_bias"], M["ddt_bias"] = g["ddt"].sum(0), M["ddt"].sum(0)
    return {k: (g[k], M[k]) for k in g}


# ------------------------------------------------------------------------ norms

def norm_before(x, w, res=None, scale=None, eps=1e-5):
    """out, r and their magnitudes."""
    sx = x if scale is None else x * scale
    r = sx if res is None else res + sx
    mr = sx.abs() + (0 if res is None else res.abs())
    rstd = (r.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    out = r * rstd * w
    # an error of r moves the mean by at most as much, relatively, as the row's largest relative weight
    mo = (mr + r.abs() * (r.abs() * mr).mean(1, keepdim=True) * rstd ** 2) * rstd * w.abs()
    return out, r, mo, mr


def norm_before_bwd(r, w, dout, dres=None, x=None, scale=None, eps=1e-5):
    rstd = (r.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    n, dn = r * rstd, dout * w
    dr = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    m = rstd * (dn.abs() + 2 * n.abs() * (dn * n).abs().mean(1, keepdim=True))
    if dres is not None:
        dr, m = dr + dres, m + dres.abs()
    s = 1.0 if scale is None else scale
    out = dict(dresidual=(dr, m), dx=(dr * s, m * abs(s) if scale is None else m * scale.abs()),
               dweight=((dout * n).sum(0), (dout * n).abs().sum(0)))
    if scale is not None:
        out["dscale"] = ((dr * x).sum(0), (m * x.abs()).sum(0))
    return out


def _groups(v, G):
    return v.unflatten(1, (G, -1))


def norm_after(y, z, w, res=None, scale=None, G=1, norm_first=False, eps=1e-5):
    gate = torch.ones_like(y) if z is None else silu(z)
    v = y if norm_first else y * gate
    rstd = (_groups(v, G).pow(2).mean(2, keepdim=True) + eps).rsqrt()
    n = (_groups(v, G) * rstd).flatten(1) * w
    out = n * gate if norm_first else n
    out = out if scale is None else out * scale
    mag = 3 * out.abs() + (0 if res is None else res.abs())
    return (out if res is None else out + res), mag


def norm_after_bwd(y, z, w, dout, scale=None, G=1, norm_first=False, eps=1e-5):
    gate, dgate = (torch.ones_like(y), torch.zeros_like(y)) if z is None else (silu(z), dsilu(z))
    # silu' = s (1 + z (1 - s)): its terms, for the cancellation near its zero
    mgate = torch.zeros_like(y) if z is None else torch.sigmoid(z) * (1 + z.abs())
    v = y if norm_first else y * gate
    rstd = (_groups(v, G).pow(2).mean(2, keepdim=True) + eps).rsqrt()
    n = (_groups(v, G) * rstd).flatten(1)
    dg = dout if scale is None else dout * scale
    dm = dg * gate if norm_first else dg
    dn = _groups(dm * w, G)
    mean = (dn * _groups(n, G)).mean(2, keepdim=True)
    mmean = (dn * _groups(n, G)).abs().mean(2, keepdim=True)
    dv = (rstd * (dn - _groups(n, G) * mean)).flatten(1)
    mv = (rstd * (dn.abs() + 2 * _groups(n, G).abs() * mmean)).flatten(1)
    if norm_first:
        dy, my, dz, mz = dv, mv, dg * n * w * dgate, (dg * n * w).abs() * mgate
    else:
        dy, my, dz, mz = dv * gate, mv * gate.abs(), dv * y * dgate, mv * y.abs() * mgate
    out = dict(dy=(dy, my), dz=(dz, mz), dweight=((dm * n).sum(0), (dm * n).abs().sum(0)))
    if scale is not None:
        gated = n * w * (gate if norm_first else 1.0)
        out["dscale"] = ((dout * gated).sum(0), (dout * gated).abs().sum(0))
    return out
