"""What lies between the matrix products of a selective state space block: the
short causal convolution, the selective scan with its gate, and the norms
before and after, for ragged prompts, for single tokens and for training.

``run`` computes one pass of a case, in elementary torch operations or, with
``own``, through the library's entry points.  Tokens of several sequences are
packed one after another; ``cu`` holds the sequences' boundaries.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    """Four operators (conv, scan, norm before, norm after), each in its forms."""
    ragged = "1,730,2048,64,3,1500,129,2047,512,31,900,1203"
    return [
        # decoding: the conv of one new token for 64 sequences, BitMamba-1B widths
        dict(name="conv-token-64seq", op="conv", form="token", io="bf16", seqs=64, slots=80, xc=4096, bc=128, width=4),
        # serving: the conv of twelve prompts of a batch, some continued, BitMamba-1B widths
        dict(name="conv-prompts-bf16", op="conv", form="prompts", io="bf16", lens=ragged, slots=16, xc=4096, bc=128, width=4),
        # training in float32: packed documents, forward and gradient, Mamba-1 widths
        dict(name="conv-train-f32", op="conv", form="train", io="f32", lens="4096,1000,77,2819,1,4100,3391", xc=1024, bc=0, width=4),
        # decoding one sequence: latency
        dict(name="scan-token-1seq", op="scan", form="token", io="bf16", seqs=1, slots=4, channels=1024, groups=1, dstate=16),
        # decoding a large batch: the states' bandwidth
        dict(name="scan-token-256seq", op="scan", form="token", io="bf16", seqs=256, slots=300, channels=4096, groups=1, dstate=16),
        # serving: the scan of twelve prompts, some continued
        dict(name="scan-prompts-bf16", op="scan", form="prompts", io="bf16", lens=ragged, slots=16, channels=1024, groups=1, dstate=16),
        # one long prompt, float32
        dict(name="scan-long-f32", op="scan", form="prompts", io="f32", lens="16384", slots=1, channels=2048, groups=1, dstate=16),
        # training: the Mamba-50M card's batch and context, forward and gradient
        dict(name="scan-train-64x512", op="scan", form="train", io="bf16", lens=",".join(["512"] * 64), channels=1024, groups=1, dstate=16),
        # decoding: the norm before a block for eight rows, float32 residual stream
        dict(name="before-token-8rows", op="before", form="forward", io="bf16", res="f32", rows=8, width=2048, scaled=False),
        # training: the norm before a block, forward and gradient
        dict(name="before-train-16k", op="before", form="train", io="bf16", res="f32", rows=16384, width=2048, scaled=True),
        # an odd batch of prompts in float32, gate after the norm, residual and scale
        dict(name="after-prompts-f32", op="after", form="forward", io="f32", rows=1023, width=1000, groups=1, gate="after", scaled=True),
        # training: the gated norm of a Mamba-2 mixer with eight groups, forward and gradient
        dict(name="after-train-8k", op="after", form="train", io="bf16", rows=8192, width=4096, groups=8, gate="before", scaled=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total, seqs):
    """seqs lengths, some of one token, of about total tokens in all."""
    w = [rng.expovariate(1.0) + 1e-3 for _ in range(seqs)]
    return ",".join(str(max(1, int(total * v / sum(w)))) for v in w)


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "before", "after"])
    io = rng.choice(["bf16", "f32"])
    if op in ("conv", "scan"):
        form = rng.choice(["token", "prompts", "train"])
        case = dict(op=op, form=form, io=io)
        if form == "token":
            n = _log(rng, 1, 256)
            case.update(seqs=n, slots=n + rng.randint(0, 40))
        else:
            seqs = _log(rng, 1, 64)
            top = 9000 if op == "conv" else (9000 if form == "prompts" else 8000)
            case.update(lens=_lens(rng, _log(rng, 16 * seqs, top), seqs))
            if form == "prompts":
                case.update(slots=seqs + rng.randint(0, 5))
        if op == "conv":
            case.update(xc=_log(rng, 64, 4096), bc=rng.choice([0, 16, 64, 128]), width=rng.randint(2, 4))
        else:
            groups = rng.choice([1, 1, 2])
            case.update(channels=groups * _log(rng, 64, 2048 // groups), groups=groups, dstate=rng.choice([4, 8, 16, 16, 32]))
            if case["dstate"] == 32 and form != "token":
                case["channels"] = groups * _log(rng, 64, 1024 // groups)
        return case
    form = rng.choice(["forward", "train"])
    groups = rng.choice([1, 1, 2, 8]) if op == "after" else 1
    case = dict(op=op, form=form, io=io, rows=_log(rng, 1, 8192), width=groups * _log(rng, 64, 4096 // groups), scaled=rng.random() < 0.5)
    if op == "before":
        case.update(res=rng.choice([io, "f32"]))
    else:
        case.update(groups=groups, gate=rng.choice(["before", "after"]))
    return case


# ------------------------------------------------------------------- inputs

def _split(case):
    return [int(v) for v in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    io, f32 = IO[case["io"]], torch.float32

    def randn(*shape, dtype=f32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case)
    if case["op"] in ("conv", "scan"):
        if case["form"] == "token":
            n = case["seqs"]
        else:
            lens = _split(case)
            n = sum(lens)
            s["cu"] = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
            s["longest"] = max(lens)
        if case["form"] != "train":
            rows = case["seqs"] if case["form"] == "token" else len(lens)
            s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:rows].to(torch.int32)
            s["has_init"] = torch.rand(rows, generator=g, device="cuda") < 0.5
    if case["op"] == "conv":
        c = case["xc"] + 2 * case["bc"]
        # a slice of the input projection's output, which holds the gate beside it
        s["xbc"] = randn(n, c + case["xc"], dtype=io)[:, case["xc"]:]
        s["weight"] = randn(c, case["width"], scale=case["width"] ** -0.5)
        s["bias"] = randn(c, scale=0.1)
        if case["form"] == "train":
            s["dout"] = [randn(n, w, dtype=io) for w in (case["xc"], case["bc"], case["bc"])]
        else:
            s["state"] = randn(case["slots"], c, case["width"] - 1, dtype=io)
    elif case["op"] == "scan":
        d, N, G = case["channels"], case["dstate"], case["groups"]
        s["x"] = randn(n, d, dtype=io)
        s["z"] = randn(n, 2 * d, dtype=io)[:, d:]
        rank = 8 * ((d + 127) // 128)
        xdbl = randn(n, rank + 2 * G * N, dtype=io)
        s["B"] = xdbl[:, rank:rank + G * N].unflatten(1, (G, N))
        s["C"] = xdbl[:, rank + G * N:].unflatten(1, (G, N))
        s["dt"] = randn(n, d, dtype=io, scale=0.5)
        step = torch.exp(uniform(math.log(1e-3), math.log(0.1), d))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=f32) * uniform(0.8, 1.2, d, N)
        s["D"] = randn(d)
        if case["form"] == "train":
            s["dy"] = randn(n, d, dtype=io)
        else:
            s["state"] = randn(case["slots"], d, N)
    elif case["op"] == "before":
        r, w = case["rows"], case["width"]
        s["x"], s["residual"] = randn(r, w, dtype=io), randn(r, w, dtype=IO[case["res"]], scale=3.0)
        s["weight"] = 1.0 + randn(w, scale=0.1)
        s["scale"] = uniform(0.1, 1.0, w) if case["scaled"] else None
        if case["form"] == "train":
            s["dout"], s["dres"] = randn(r, w, dtype=io), randn(r, w, dtype=IO[case["res"]])
    else:
        r, w = case["rows"], case["width"]
        s["y"], s["z"] = randn(r, w, dtype=io), randn(r, 2 * w, dtype=io)[:, :w]
        s["weight"] = 1.0 + randn(w, scale=0.1)
        s["scale"] = uniform(0.1, 1.0, w) if case["scaled"] else None
        s["residual"] = randn(r, w, dtype=io) if case["scaled"] else None
        if case["form"] == "train":
            s["dout"] = randn(r, w, dtype=io)
    return s


# -------------------------------------------------------------- plain forms

def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _where(s, n):
    """Of each packed token: its sequence, its sequence's first token and end."""
    t = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    return t, seq, s["cu"][seq].long(), s["cu"][seq + 1].long()


def _conv_token(s):
    case, slots = s["case"], s["slots"].long()
    old = s["state"][slots].float()
    win = torch.cat([old, s["xbc"].float()[:, :, None]], 2)
    out = _silu((win * s["weight"]).sum(2) + s["bias"]).to(s["xbc"].dtype)
    s["state"][slots] = win[:, :, 1:].to(s["state"].dtype)
    return list(out.split([case["xc"], case["bc"], case["bc"]], 1)) + [s["state"]]


def _taps(s, x):
    """[tokens, K, channels]: the K inputs under each token's window."""
    K = s["case"]["width"]
    t, seq, first, _ = _where(s, x.shape[0])
    rows = t[:, None] - (K - 1) + torch.arange(K, device="cuda")
    inside = (rows >= first[:, None])[:, :, None]
    if "state" not in s:
        return torch.where(inside, x[rows.clamp(min=0)], 0.0)
    init = s["state"][s["slots"].long()].float() * s["has_init"][:, None, None]
    return torch.where(inside, x[rows.clamp(min=0)], init.transpose(1, 2)[seq[:, None], (rows - first[:, None] + K - 1).clamp(0, K - 2)])


def _conv_prompts(s):
    case, K = s["case"], s["case"]["width"]
    x = s["xbc"].float()
    taps = _taps(s, x)
    out = _silu((taps * s["weight"].T).sum(1) + s["bias"]).to(s["xbc"].dtype)
    s["state"][s["slots"].long()] = taps[s["cu"][1:].long() - 1][:, 1:].transpose(1, 2).to(s["state"].dtype)
    return list(out.split([case["xc"], case["bc"], case["bc"]], 1)) + [s["state"]]


def _conv_train(s):
    case, K, io = s["case"], s["case"]["width"], s["xbc"].dtype
    x = s["xbc"].float()
    taps = _taps(s, x)
    pre = (taps * s["weight"].T).sum(1) + s["bias"]
    dpre = torch.cat(s["dout"], 1).float() * _dsilu(pre)
    t, _, _, end = _where(s, x.shape[0])
    rows = t[:, None] + (K - 1) - torch.arange(K, device="cuda")
    later = torch.where((rows < end[:, None])[:, :, None], dpre[rows.clamp(max=x.shape[0] - 1)], 0.0)
    return list(_silu(pre).to(io).split([case["xc"], case["bc"], case["bc"]], 1)) + [
        (later * s["weight"].T).sum(1).to(io), (dpre[:, None] * taps).sum(0).T.contiguous(), dpre.sum(0)]


def _spread(v, d):
    """[tokens, groups, dstate] as [tokens, channels, dstate] in 32 bits."""
    return v.float().repeat_interleave(d // v.shape[1], 1)


def _scan_token(s):
    slots, d = s["slots"].long(), s["case"]["channels"]
    x, delta = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[:, :, None] * s["A"]) * s["state"][slots] + (delta * x)[:, :, None] * _spread(s["B"], d)
    s["state"][slots] = h
    y = (h * _spread(s["C"], d)).sum(2) + s["D"] * x
    return [(y * _silu(s["z"].float())).to(s["x"].dtype), s["state"]]


def _recurrence(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling."""
    n = 1
    while n < longest:
        b = torch.cat([b[:n], b[n:] + a[n:] * b[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return b


def _scan_parts(s):
    d = s["case"]["channels"]
    x, raw = s["x"].float(), s["dt"].float() + s["dt_bias"]
    delta = _softplus(raw)
    a = torch.exp(delta[:, :, None] * s["A"])
    B, C = _spread(s["B"], d), _spread(s["C"], d)
    b = (delta * x)[:, :, None] * B
    start = s["cu"][:-1].long()
    if "state" in s:
        b[start] += a[start] * (s["state"][s["slots"].long()] * s["has_init"][:, None, None])
    a[start] = 0.0
    return x, raw, delta, a, B, C, _recurrence(a, b, s["longest"])


def _scan_prompts(s):
    x, _, _, _, _, C, h = _scan_parts(s)
    y = ((h * C).sum(2) + s["D"] * x) * _silu(s["z"].float())
    s["state"][s["slots"].long()] = h[s["cu"][1:].long() - 1]
    return [y.to(s["x"].dtype), s["state"]]


def _scan_train(s):
    io, G, d = s["x"].dtype, s["case"]["groups"], s["case"]["channels"]
    x, raw, delta, a, B, C, h = _scan_parts(s)
    z, dy = s["z"].float(), s["dy"].float()
    ungated = (h * C).sum(2) + s["D"] * x
    dz, dyp = dy * ungated * _dsilu(z), dy * _silu(z)
    g = _recurrence(torch.cat([a[1:], torch.zeros_like(a[:1])]).flip(0), (dyp[:, :, None] * C).flip(0), s["longest"]).flip(0)
    q = g * (a * torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
    du = (g * B).sum(2)
    ddt = (x * du + (q * s["A"]).sum(2)) * torch.sigmoid(raw)
    per_group = lambda v: v.unflatten(1, (G, d // G)).sum(2).to(io)  # noqa: E731
    return [(ungated * _silu(z)).to(io), (delta * du + s["D"] * dyp).to(io), ddt.to(io), (delta[:, :, None] * q).sum(0),
            per_group((delta * x)[:, :, None] * g), per_group(dyp[:, :, None] * h), (dyp * x).sum(0), dz.to(io), ddt.sum(0)]


def _before(s):
    io, res = s["x"].dtype, s["residual"].dtype
    x, scale = s["x"].float(), 1.0 if s["scale"] is None else s["scale"]
    r = s["residual"].float() + scale * x
    out = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["weight"]
    outputs = [out.to(io), r.to(res)]
    if "dout" not in s:
        return outputs
    r, dout = outputs[1].float(), s["dout"].float()  # the gradient works from the residual that was stored
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n, dn = r * rstd, dout * s["weight"]
    dr = rstd * (dn - n * (dn * n).mean(1, keepdim=True)) + s["dres"].float()
    outputs += [(scale * dr).to(io), dr.to(res), (dout * n).sum(0)]
    return outputs if s["scale"] is None else outputs + [(dr * x).sum(0)]


def _after(s):
    io, G = s["y"].dtype, s["case"]["groups"]
    y, z, w = s["y"].float(), s["z"].float(), s["weight"]
    first = s["case"]["gate"] == "before"
    v = (y * _silu(z) if first else y).unflatten(1, (G, -1))
    rstd = torch.rsqrt((v * v).mean(2, keepdim=True) + EPS)
    n = v * rstd
    normed = n.flatten(1) * w
    gated = normed if first else normed * _silu(z)
    out = gated if s["scale"] is None else s["residual"].float() + s["scale"] * gated
    if "dout" not in s:
        return [out.to(io)]
    dout = s["dout"].float()
    dgated = dout if s["scale"] is None else dout * s["scale"]
    dnormed = dgated if first else dgated * _silu(z)
    dn = (dnormed * w).unflatten(1, (G, -1))
    dv = (rstd * (dn - n * (dn * n).mean(2, keepdim=True))).flatten(1)
    dy, dz = (dv * _silu(z), dv * y * _dsilu(z)) if first else (dv, dgated * normed * _dsilu(z))
    outputs = [out.to(io), dy.to(io), dz.to(io), (dnormed * n.flatten(1)).sum(0)]
    return outputs if s["scale"] is None else outputs + [(dout * gated).sum(0)]


# ------------------------------------------------------- the library's calls

def _own(s):
    import selective_state_space_22_b200 as ssd

    case, form = s["case"], s["case"]["form"]
    if case["op"] == "conv":
        widths = dict(x_channels=case["xc"], bc_channels=case["bc"])
        if form == "token":
            return list(ssd.ssd_conv1d_update(s["state"], s["xbc"], s["weight"], s["bias"], slots=s["slots"], **widths)) + [s["state"]]
        if form == "prompts":
            return list(ssd.ssd_conv1d_varlen(s["xbc"], s["weight"], s["bias"], s["cu"], conv_state=s["state"], slots=s["slots"], has_init=s["has_init"], **widths)) + [s["state"]]
        out = ssd.ssd_conv1d_varlen(s["xbc"], s["weight"], s["bias"], s["cu"], **widths)
        g = ssd.ssd_conv1d_bwd(s["xbc"], s["weight"], s["bias"], s["cu"], *s["dout"])
        return list(out) + [g["dxbc"], g["dweight"], g["dbias"]]
    if case["op"] == "scan":
        if form == "token":
            y = ssd.ssd_selective_state_update(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], slots=s["slots"])
            return [y, s["state"]]
        if form == "prompts":
            y, _ = ssd.ssd_selective_scan_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["D"], s["z"], s["dt_bias"], state=s["state"],
                                                 slots=s["slots"], has_init=s["has_init"])
            return [y, s["state"]]
        y, chunks = ssd.ssd_selective_scan_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["D"], s["z"], s["dt_bias"], return_chunk_states=True)
        g = ssd.ssd_selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["dy"], chunks, s["D"], s["z"], s["dt_bias"])
        return [y] + [g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")]
    if case["op"] == "before":
        out, r = ssd.ssd_residual_rmsnorm(s["x"], s["weight"], s["residual"], s["scale"], eps=EPS)
        if form == "forward":
            return [out, r]
        g = ssd.ssd_residual_rmsnorm_bwd(r, s["weight"], s["dout"], s["dres"], s["x"], s["scale"], eps=EPS)
        return [out, r, g["dx"], g["dresidual"], g["dweight"]] + ([] if s["scale"] is None else [g["dscale"]])
    kind = dict(ngroups=case["groups"], eps=EPS, norm_before_gate=case["gate"] == "after")
    out = ssd.ssd_gated_rmsnorm(s["y"], s["z"], s["weight"], s["residual"], s["scale"], **kind)
    if form == "forward":
        return [out]
    g = ssd.ssd_gated_rmsnorm_bwd(s["y"], s["z"], s["weight"], s["dout"], s["scale"], **kind)
    return [out, g["dy"], g["dz"], g["dweight"]] + ([] if s["scale"] is None else [g["dscale"]])


PLAIN = {("conv", "token"): _conv_token, ("conv", "prompts"): _conv_prompts, ("conv", "train"): _conv_train,
         ("scan", "token"): _scan_token, ("scan", "prompts"): _scan_prompts, ("scan", "train"): _scan_train,
         ("before", "forward"): _before, ("before", "train"): _before, ("after", "forward"): _after, ("after", "train"): _after}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"], state["case"]["form"]](state)


# --------------------------------------------------------------------- work

def work(case):
    e = 2 if case["io"] == "bf16" else 4
    train = case["form"] == "train"
    if case["op"] in ("conv", "scan"):
        n = case["seqs"] if case["form"] == "token" else sum(_split(case))
        seqs = case["seqs"] if case["form"] == "token" else len(_split(case))
    if case["op"] == "conv":
        c, K = case["xc"] + 2 * case["bc"], case["width"]
        if train:  # input, its output, the output's gradient, the input's gradient
            return {"bytes": 4 * n * c * e + 8 * c * (K + 1), "flops": n * c * (6 * K + 12)}
        return {"bytes": 2 * n * c * e + 2 * seqs * c * (K - 1) * e + 4 * c * (K + 1), "flops": n * c * (2 * K + 4)}
    if case["op"] == "scan":
        d, N, G = case["channels"], case["dstate"], case["groups"]
        if train:  # x, dt, z, dy read; y, dx, ddt, dz written; B, C and their gradients
            return {"bytes": n * (8 * d + 4 * G * N) * e + 8 * d * (N + 2), "flops": n * d * (22 * N + 40)}
        return {"bytes": n * (4 * d + 2 * G * N) * e + 8 * seqs * d * N + 4 * d * (N + 2), "flops": n * d * (6 * N + 12)}
    m = case["rows"] * case["width"]
    if case["op"] == "before":
        r = 2 if case["res"] == "bf16" else 4
        if train:  # x, residual, both gradients read; out, residual, both gradients written
            return {"bytes": m * (4 * e + 4 * r) + 12 * case["width"], "flops": 20 * m}
        return {"bytes": m * (2 * e + 2 * r) + 4 * case["width"], "flops": 6 * m}
    if train:  # y, z, dout (and residual) read; out, dy, dz written
        return {"bytes": m * (7 if case["scaled"] else 6) * e + 12 * case["width"], "flops": 32 * m}
    return {"bytes": m * (4 if case["scaled"] else 3) * e + 4 * case["width"], "flops": 12 * m}


# ------------------------------------------- the definitions, in 64 bits

def _each(s):
    """(first, end, sequence) of every packed sequence."""
    cu = s["cu"].tolist()
    return [(cu[i], cu[i + 1], i) for i in range(len(cu) - 1)]


def _exact_conv(s):
    case, K = s["case"], s["case"]["width"]
    f = torch.nn.functional
    x, w, b = s["xbc"].double(), s["weight"].double(), s["bias"].double()
    pieces = [case["xc"], case["bc"], case["bc"]]
    if case["form"] == "token":
        spans = [(i, i + 1, i) for i in range(x.shape[0])]
        init = s["state"].double()[s["slots"].long()]
    else:
        spans = _each(s)
        init = torch.zeros(len(spans), x.shape[1], K - 1, dtype=torch.float64, device="cuda")
        if case["form"] == "prompts":
            init[s["has_init"]] = s["state"].double()[s["slots"].long()][s["has_init"]]
    if case["form"] == "token":
        win = torch.cat([init, x[:, :, None]], 2)
        out = f.silu(torch.einsum("bck,ck->bc", win, w) + b)
        last = win[:, :, 1:]
    else:
        w.requires_grad_(), b.requires_grad_(), x.requires_grad_()
        outs, lasts = [], []
        for lo, hi, i in spans:
            seq = torch.cat([init[i], x[lo:hi].T], 1)
            outs.append(f.silu(f.conv1d(seq[None], w[:, None], b, groups=w.shape[0])[0]).T)
            lasts.append(seq[:, -(K - 1):])
        out, last = torch.cat(outs), torch.stack(lasts)
    if case["form"] == "train":
        grads = torch.autograd.grad(out, (x, w, b), torch.cat(s["dout"], 1).double())
        return list(out.detach().split(pieces, 1)) + list(grads)
    state = s["state"].double()
    state[s["slots"].long()] = last.detach()
    return list(out.detach().split(pieces, 1)) + [state]


def _exact_scan(s):
    case = s["case"]
    f, d, N, G, train = torch.nn.functional, case["channels"], case["dstate"], case["groups"], case["form"] == "train"
    spans = [(i, i + 1, i) for i in range(case["seqs"])] if case["form"] == "token" else _each(s)
    longest = max(hi - lo for lo, hi, _ in spans)
    lo = torch.tensor([v[0] for v in spans], device="cuda")
    live = torch.arange(longest, device="cuda")[:, None] < torch.tensor([v[1] - v[0] for v in spans], device="cuda")
    rows = torch.where(live, lo + torch.arange(longest, device="cuda")[:, None], 0)  # [time, sequence]
    raw = s["dt"].double() + s["dt_bias"].double()
    delta = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    x, A, D = s["x"].double(), s["A"].double(), s["D"].double()
    B, C = s["B"].double(), s["C"].double()
    of = torch.arange(d, device="cuda") // (d // G)
    h = torch.zeros(len(spans), d, N, dtype=torch.float64, device="cuda")
    if not train:
        init = s["state"].double()[s["slots"].long()]
        h = init if case["form"] == "token" else init * s["has_init"][:, None, None]
    pre = torch.zeros_like(x)
    kept = torch.empty(longest, *h.shape, dtype=torch.float64, device="cuda") if train else None
    for t in range(longest):
        on, r = live[t], rows[t]
        new = torch.exp(delta[r][:, :, None] * A) * h + (delta[r] * x[r])[:, :, None] * B[r][:, of]
        h = torch.where(on[:, None, None], new, h)
        if train:
            kept[t] = h
        pre[r[on]] = ((h * C[r][:, of]).sum(2) + D * x[r])[on]
    z = s["z"].double()
    y = pre * f.silu(z)
    if not train:
        state = s["state"].double()
        state[s["slots"].long()] = h
        return [y, state]
    dy, p = s["dy"].double(), torch.sigmoid(z)
    dz, dyp = dy * pre * p * (1 + z * (1 - p)), dy * z * p
    dx, ddelta, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A)
    dB, dC = torch.zeros_like(B), torch.zeros_like(C)
    carry = torch.zeros_like(h)
    for t in reversed(range(longest)):
        on, r = live[t], rows[t]
        o = on[:, None, None]
        a = torch.exp(delta[r][:, :, None] * A)
        before = kept[t - 1] if t else torch.zeros_like(h)
        g = torch.where(o, dyp[r][:, :, None] * C[r][:, of] + carry, 0.0)
        q = g * a * before
        du = (g * B[r][:, of]).sum(2)
        dA += (delta[r][:, :, None] * q).sum(0)
        k = r[on]
        dx[k] = (delta[r] * du + D * dyp[r])[on]
        ddelta[k] = (x[r] * du + (q * A).sum(2))[on]
        dB[k] = ((delta[r] * x[r])[:, :, None] * g).unflatten(1, (G, -1)).sum(2)[on]
        dC[k] = (dyp[r][:, :, None] * kept[t]).unflatten(1, (G, -1)).sum(2)[on]
        carry = torch.where(o, a * g, carry)
    ddt = ddelta * torch.sigmoid(raw)
    return [y, dx, ddt, dA, dB, dC, (dyp * x).sum(0), dz, ddt.sum(0)]


def _exact_norm(s):
    case = s["case"]
    f, train = torch.nn.functional, case["form"] == "train"
    w = s["weight"].double().requires_grad_()
    scale = None if s["scale"] is None else s["scale"].double().requires_grad_()
    times = 1.0 if scale is None else scale

    def norm(v, groups):
        v = v.unflatten(1, (groups, -1))
        return (v / torch.sqrt(v.pow(2).mean(2, keepdim=True) + EPS)).flatten(1) * w

    if case["op"] == "before":
        x = s["x"].double()
        r = s["residual"].double() + (1.0 if scale is None else scale.detach()) * x
        outputs = [norm(r, 1).detach(), r]
        if not train:
            return outputs
        stored = r.to(s["residual"].dtype).double().requires_grad_()
        dr, dw = torch.autograd.grad(norm(stored, 1), (stored, w), s["dout"].double())
        dr = dr + s["dres"].double()
        outputs += [(dr * times).detach(), dr, dw]
        return outputs if scale is None else outputs + [(dr * x).sum(0)]
    y, z = s["y"].double().requires_grad_(), s["z"].double().requires_grad_()
    out = norm(y * f.silu(z), case["groups"]) if case["gate"] == "before" else norm(y, case["groups"]) * f.silu(z)
    if scale is not None:
        out = s["residual"].double() + scale * out
    if not train:
        return [out.detach()]
    wrt = (y, z, w) if scale is None else (y, z, w, scale)
    return [out.detach()] + list(torch.autograd.grad(out, wrt, s["dout"].double()))


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan}.get(case["op"], _exact_norm)(s)
