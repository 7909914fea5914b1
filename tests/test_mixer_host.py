"""The mixer-block operators without a GPU: the C ABI's refusals (nothing is
launched), the binding's checks, and the 64-bit formulas the GPU tests compare with
against automatic differentiation and against differences."""
import ctypes

import pytest
import torch

import mixer_ref as ref
import selective_state_space_22_b200 as ssd
from selective_state_space_22_b200 import build as ssd_build
from selective_state_space_22_b200.mixer import _SelArgs

FAKE = 1 << 20  # 16-byte aligned, never dereferenced
OFF = FAKE + 4
BAD, UNSUP, WORK = ssd.SSD_ERR_INVALID_ARG, ssd.SSD_ERR_UNSUPPORTED, ssd.SSD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load_library()


def call(fn, names, defaults, over):
    args = dict(defaults, **over)
    return fn(*[args[k] for k in names.split()])


CONV = dict(xbc=FAKE, ld=96, w=FAKE, b=None, cu=FAKE, st=None, slots=None, has=None, xo=FAKE, bo=FAKE, co=FAKE, io=0, n=10,
            nseq=2, nslots=0, cx=64, cb=16, K=4, silu=1, stream=None)


@pytest.mark.parametrize("over,status,msg", [
    (dict(xbc=None), BAD, "non-null"), (dict(w=None), BAD, "non-null"), (dict(xo=None), BAD, "non-null"),
    (dict(bo=None), BAD, "non-null"), (dict(cu=None), BAD, "non-null"), (dict(io=3), BAD, "io_dtype"),
    (dict(cx=0), BAD, "x_channels"), (dict(K=0), UNSUP, "width"), (dict(K=9), UNSUP, "width"), (dict(ld=95), BAD, "below"),
    (dict(n=-1), BAD, ">= 0"), (dict(nseq=-1), BAD, ">= 0"), (dict(w=OFF), BAD, "aligned"), (dict(xbc=FAKE + 2), BAD, "aligned"),
    (dict(st=FAKE, nslots=1), BAD, "slots"), (dict(st=OFF, nslots=2), BAD, "aligned"), (dict(cx=1 << 20), UNSUP, "channels"),
])
def test_conv_varlen_refusals(lib, over, status, msg):
    if over.get("cx") == 1 << 20:
        over = dict(over, ld=1 << 22)
    assert call(lib.ssd_conv1d_varlen, "xbc ld w b cu st slots has xo bo co io n nseq nslots cx cb K silu stream", CONV, over) == status
    assert msg in ssd.ssd_last_error()


@pytest.mark.parametrize("over,status,msg", [
    (dict(st=None), BAD, "non-null"), (dict(n=-1), BAD, "batch"), (dict(n=65536, nslots=65536), UNSUP, "batch"), (dict(nslots=9), BAD, "slots"),
    (dict(xo=OFF), BAD, "aligned"), (dict(K=9), UNSUP, "width"),
])
def test_conv_update_refusals(lib, over, status, msg):
    base = dict(CONV, st=FAKE, nslots=10)
    assert call(lib.ssd_conv1d_update, "st slots xbc ld w b xo bo co io n nslots cx cb K silu stream", base, over) == status
    assert msg in ssd.ssd_last_error()


@pytest.mark.parametrize("over,status,msg", [
    (dict(xbc=None), BAD, "non-null"), (dict(dw=None), BAD, "non-null"), (dict(dx=None), BAD, "non-null"), (dict(co=None), BAD, "non-null"),
    (dict(ws=None), WORK, "needed"), (dict(wsb=8), WORK, "needed"), (dict(dx=OFF), BAD, "aligned"), (dict(ws=OFF), BAD, "aligned"),
    (dict(cu=None), BAD, "non-null"),
])
def test_conv_bwd_refusals(lib, over, status, msg):
    base = dict(CONV, dx=FAKE, dw=FAKE, db=None, ws=FAKE, wsb=1 << 30)
    assert call(lib.ssd_conv1d_bwd, "xbc ld w b cu xo bo co dx dw db io n nseq cx cb K silu ws wsb stream", base, over) == status
    assert msg in ssd.ssd_last_error()


def sel_args(**over):
    a = _SelArgs()
    base = dict(x=FAKE, dt=FAKE, z=None, B=FAKE, C=FAKE, A=FAKE, D=None, dt_bias=None, x_stride=64, dt_stride=64, z_stride=64,
                b_stride=16, c_stride=16, io_dtype=0, softplus=1, channels=64, ngroups=1, dstate=16)
    for k, v in dict(base, **over).items():
        setattr(a, k, v)
    return a


SEL_REFUSALS = [
    (dict(x=None), BAD, "non-null"), (dict(A=None), BAD, "non-null"), (dict(C=None), BAD, "non-null"), (dict(dt=FAKE + 2), BAD, "aligned"),
    (dict(A=OFF), BAD, "aligned"), (dict(io_dtype=2), BAD, "io_dtype"), (dict(ngroups=3), BAD, "divide"), (dict(channels=0), BAD, "> 0"),
    (dict(dstate=65), UNSUP, "dstate"), (dict(x_stride=63), BAD, "below"), (dict(z=FAKE, z_stride=1), BAD, "below"),
    (dict(b_stride=15), BAD, "below"), (dict(channels=1 << 20, x_stride=1 << 20, dt_stride=1 << 20), UNSUP, "grid"),
]


@pytest.mark.parametrize("over,status,msg", SEL_REFUSALS)
def test_scan_refusals(lib, over, status, msg):
    a = sel_args(**over)
    for st in (lib.ssd_selective_scan_varlen(a, FAKE, None, None, None, None, FAKE, 10, 2, 0, FAKE, 1 << 30, None),
               lib.ssd_selective_state_update(a, FAKE, None, FAKE, 10, 10, None),
               lib.ssd_selective_scan_bwd(a, FAKE, FAKE, FAKE, *[FAKE] * 8, 10, 2, FAKE, 1 << 40, None)):
        assert st == status and msg in ssd.ssd_last_error()


def test_scan_refusals_of_each_call(lib):
    a = sel_args()
    varlen = lambda *, cu=FAKE, st=None, y=FAKE, n=10, nseq=2, nslots=0, kept=None, ws=FAKE: lib.ssd_selective_scan_varlen(  # noqa: E731
        a, cu, st, None, None, kept, y, n, nseq, nslots, ws, 1 << 20, None)
    assert varlen(cu=None) == BAD and varlen(y=None) == BAD and varlen(n=-1) == BAD and varlen(y=OFF) == BAD
    assert varlen(st=FAKE, nslots=1) == BAD and "slots" in ssd.ssd_last_error()
    assert varlen(n=(1 << 31) - 1) == UNSUP
    assert lib.ssd_selective_scan_varlen(None, FAKE, None, None, None, None, FAKE, 10, 2, 0, FAKE, 1 << 30, None) == BAD
    update = lambda *, st=FAKE, y=FAKE, n=10, nslots=10: lib.ssd_selective_state_update(a, st, None, y, n, nslots, None)  # noqa: E731
    assert update(st=None) == BAD and update(y=None) == BAD and update(n=-1) == BAD and update(n=65536) == UNSUP and update(nslots=9) == BAD

    def bwd(k=None, v=None, ws=FAKE, wsb=1 << 30):
        p = dict(cu=FAKE, dy=FAKE, kept=FAKE, dx=FAKE, ddt=FAKE, dz=None, dB=FAKE, dC=FAKE, dA=FAKE, dD=None, dbias=None)
        if k:
            p[k] = v
        return lib.ssd_selective_scan_bwd(a, *p.values(), 10, 2, ws, wsb, None)

    for k in ("cu", "dy", "kept", "dx", "ddt", "dB", "dC", "dA"):
        assert bwd(k) == BAD and "non-null" in ssd.ssd_last_error(), k
    assert bwd("dx", OFF) == BAD and bwd(ws=None) == WORK and bwd(wsb=64) == WORK
    assert varlen(n=1 << 20, ws=None) == WORK and varlen(n=1 << 20) == WORK and varlen(ws=OFF) == BAD
    assert lib.ssd_selective_scan_workspace_size(1 << 20, 2, 64, 16) > 1 << 20
    assert lib.ssd_selective_scan_workspace_size(64 * 512, 64, 1024, 16) == 0
    assert lib.ssd_selective_scan_chunk_states(300, 3) == 300 // 8 + 3 and lib.ssd_selective_scan_chunk_states(-1, 3) == ssd.SSD_WORKSPACE_INVALID
    assert lib.ssd_selective_scan_bwd_workspace_size(10, 2, 64, 3, 16) == ssd.SSD_WORKSPACE_INVALID


def test_norm_refusals(lib):
    before = dict(x=FAKE, ldx=8, r=FAKE, ldr=8, s=None, w=FAKE, o=FAKE, ro=FAKE, io=1, rio=0, rows=4, width=8, eps=1e-5, stream=None)
    run = lambda **o: call(lib.ssd_residual_rmsnorm, " ".join(before), before, o)  # noqa: E731
    assert run(x=None) == BAD and run(w=None) == BAD and run(o=None) == BAD and run(ldx=7) == BAD and run(ldr=7) == BAD
    assert run(rows=-1) == BAD and run(width=0) == BAD and run(width=8193, ldx=9000, ldr=9000) == UNSUP and run(eps=-1.0) == BAD
    assert run(io=0, rio=1) == BAD and "residual_dtype" in ssd.ssd_last_error()
    assert run(eps=float("nan")) == BAD and run(x=FAKE + 1) == BAD and run(o=OFF) == BAD
    after = dict(y=FAKE, ldy=8, z=FAKE, ldz=8, r=None, ldr=0, s=None, w=FAKE, o=FAKE, io=1, rows=4, width=8, g=2, first=0, eps=1e-5, stream=None)
    run = lambda **o: call(lib.ssd_gated_rmsnorm, " ".join(after), after, o)  # noqa: E731
    assert run(g=3) == BAD and run(g=0) == BAD and run(y=None) == BAD and run(ldz=7) == BAD and run(r=FAKE) == BAD and run(io=2) == BAD
    b = dict(r=FAKE, ldr=8, w=FAKE, do=FAKE, dr=None, x=None, ldx=0, s=None, dx=FAKE, dri=FAKE, dw=FAKE, ds=None, io=1, rio=1, rows=4,
             width=8, eps=1e-5, ws=FAKE, wsb=1 << 20, stream=None)
    run = lambda **o: call(lib.ssd_residual_rmsnorm_bwd, " ".join(b), b, o)  # noqa: E731
    assert run(r=None) == BAD and run(dw=None) == BAD and run(s=FAKE) == BAD and run(s=FAKE, ds=FAKE) == BAD and run(dx=None, dri=None) == BAD
    assert run(ws=None) == WORK and run(wsb=8) == WORK and run(dr=OFF) == BAD
    a = dict(y=FAKE, ldy=8, z=FAKE, ldz=8, w=FAKE, do=FAKE, s=None, dy=FAKE, dz=FAKE, dw=FAKE, ds=None, io=1, rows=4, width=8, g=1,
             first=0, eps=1e-5, ws=FAKE, wsb=1 << 20, stream=None)
    run = lambda **o: call(lib.ssd_gated_rmsnorm_bwd, " ".join(a), a, o)  # noqa: E731
    assert run(y=None) == BAD and run(dz=None) == BAD and run(dw=None) == BAD and run(s=FAKE) == BAD and run(ws=None) == WORK
    assert lib.ssd_rmsnorm_bwd_workspace_size(-1, 8) == ssd.SSD_WORKSPACE_INVALID


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(4, 8)
    cu, w = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(8, 4)
    for f in (lambda: ssd.ssd_conv1d_varlen(x, w, None, cu), lambda: ssd.ssd_conv1d_update(torch.zeros(4, 8, 3), x, w),
              lambda: ssd.ssd_conv1d_bwd(x, w, None, cu, x), lambda: ssd.ssd_residual_rmsnorm(x, w[:, 0]),
              lambda: ssd.ssd_gated_rmsnorm(x, x, w[:, 0]), lambda: ssd.ssd_selective_scan_varlen(x, x, w, x[:, None], x[:, None], cu),
              lambda: ssd.ssd_selective_state_update(torch.zeros(4, 8, 4), x, x, w, x[:, None, :4], x[:, None, :4])):
        with pytest.raises(ValueError, match="CUDA"):
            f()


# ------------------------------------------------ the formulas themselves

def f64(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64)


def check(loss, inputs, grads):
    """Formula gradients against automatic ones and against central differences."""
    leaves = {k: v.clone().requires_grad_() for k, v in inputs.items()}
    auto = torch.autograd.grad(loss(**leaves), list(leaves.values()))
    g = torch.Generator().manual_seed(1)
    for (k, v), a in zip(inputs.items(), auto):
        assert torch.allclose(grads[k], a, rtol=1e-9, atol=1e-11), k
        d, h = f64(g, *v.shape), 1e-5  # the third derivative's share is h^2 of the slope
        up, down = (loss(**dict(inputs, **{k: v + s * h * d})) for s in (1, -1))
        assert abs((up - down) / (2 * h) - (a * d).sum()) <= 1e-7 * (1 + (a * d).abs().sum()), k


def test_formula_conv():
    g, cu = torch.Generator().manual_seed(0), torch.tensor([1, 3, 3, 12])
    x, w, b, up = f64(g, 13, 3), f64(g, 3, 4), f64(g, 3), f64(g, 13, 3)

    def plain(x, w, b):
        total = 0
        for lo, hi in ref.spans(cu):
            if hi > lo:
                pre = torch.nn.functional.conv1d(torch.nn.functional.pad(x[lo:hi].T, (3, 0))[None], w[:, None], b, groups=3)[0].T
                total = total + (torch.nn.functional.silu(pre) * up[lo:hi]).sum()
        return total

    out = ref.conv(x, w, b, cu, True)[0]
    assert torch.allclose((out * up)[1:12].sum(), plain(x, w, b))
    got = ref.conv_bwd(x, w, b, cu, up, True)
    check(plain, dict(x=x, w=w, b=b), dict(x=got["dxbc"][0], w=got["dweight"][0], b=got["dbias"][0]))


@pytest.mark.parametrize("softplus", [True, False])
def test_formula_scan(softplus):
    g, cu = torch.Generator().manual_seed(0), torch.tensor([0, 2, 9])
    d, G, N, n = 4, 2, 3, 9
    p = dict(x=f64(g, n, d), dt=f64(g, n, d) if softplus else f64(g, n, d).abs() * 0.1, A=-f64(g, d, N).abs(), B=f64(g, n, G, N),
             C=f64(g, n, G, N), D=f64(g, d), z=f64(g, n, d), bias=f64(g, d))
    up, of = f64(g, n, d), torch.arange(d) // (d // G)

    def loss(x, dt, A, B, C, D, z, bias):
        delta = torch.nn.functional.softplus(dt + bias) if softplus else dt + bias
        total = 0
        for lo, hi in ref.spans(cu):
            h = torch.zeros(d, N, dtype=torch.float64)
            for t in range(lo, hi):
                h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * B[t][of]
                total = total + (((h * C[t][of]).sum(1) + D * x[t]) * torch.nn.functional.silu(z[t]) * up[t]).sum()
        return total

    y = ref.sel(p["x"], p["dt"], p["A"], p["B"], p["C"], cu, p["D"], p["z"], p["bias"], softplus)[0]
    assert torch.allclose((y * up).sum(), loss(**p))
    got = ref.sel_bwd(p["x"], p["dt"], p["A"], p["B"], p["C"], cu, up, p["D"], p["z"], p["bias"], softplus)
    check(loss, p, {k: got["ddt_bias" if k == "bias" else "d" + k][0] for k in p})


def test_formula_norms():
    g = torch.Generator().manual_seed(0)
    x, r, w, s, up, up2 = f64(g, 5, 8), f64(g, 5, 8), f64(g, 8), f64(g, 8), f64(g, 5, 8), f64(g, 5, 8)

    def before(x, r, w, s):
        v = r + s * x
        return (v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-5) * w * up).sum() + (v * up2).sum()

    got = ref.norm_before_bwd(r + s * x, w, up, up2, x, s)
    check(before, dict(x=x, r=r, w=w, s=s), dict(x=got["dx"][0], r=got["dresidual"][0], w=got["dweight"][0], s=got["dscale"][0]))
    for first in (False, True):
        def after(y, z, w, s):
            gate = torch.nn.functional.silu(z)
            v = (y if first else y * gate).unflatten(1, (2, 4))
            n = (v / torch.sqrt(v.pow(2).mean(2, keepdim=True) + 1e-5)).flatten(1) * w
            return ((n * gate if first else n) * s * up).sum()

        got = ref.norm_after_bwd(x, r, w, up, s, 2, first)
        check(after, dict(y=x, z=r, w=w, s=s), dict(y=got["dy"][0], z=got["dz"][0], w=got["dweight"][0], s=got["dscale"][0]))
        assert torch.allclose((ref.norm_after(x, r, w, None, s, 2, first)[0] * up).sum(), after(x, r, w, s))
