"""The mixer-block operators on a B200 against the 64-bit formulas of mixer_ref,
element by element: packed prompts with states in slots, single tokens, gradients,
norms; odd sizes, strided rows, empty sequences, padding, malformed bounds."""
import pytest
import torch

import mixer_ref as ref
import selective_state_space_22_b200 as ssd
from mixer_ref import close, d64

pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, io=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(io).cuda()


def strided(t, pad):
    """The same values as a slice of wider rows (NaN beside them)."""
    if not pad:
        return t
    flat = t.flatten(1)
    wide = torch.full((t.shape[0], flat.shape[1] + 2 * pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, pad:pad + flat.shape[1]] = flat
    return wide[:, pad:pad + flat.shape[1]].unflatten(1, t.shape[1:])


def bounds(lens, first=0):
    return torch.tensor([first] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


# (lengths, rows before the first and behind the last sequence)
LENS = {
    "one": ([1], 0, 0), "tiny": ([1, 2, 3, 1, 1, 4], 0, 0), "empty": ([0, 5, 0, 0, 33, 0], 2, 3),
    "ragged": ([130, 1, 257, 31, 64, 2, 0, 128], 1, 5), "none": ([0], 0, 4), "long": ([700], 0, 0),
}


# ------------------------------------------------------------------ convolution

# multiply-adds of the window, the sigmoid (a few ulp of exp and divide, 16 in all) and the product
CONV_ROUNDINGS = 40


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("cx,cb,K,pad,silu,bias", [(64, 16, 4, 16, True, True), (33, 7, 4, 3, True, False),
                                                   (40, 0, 3, 0, False, True), (8, 8, 2, 8, True, True),
                                                   (17, 1, 8, 1, True, True), (24, 0, 1, 0, True, True)])
def test_conv_varlen(io, lens, cx, cb, K, pad, silu, bias):
    lens, before, behind = LENS[lens]
    io, g = IO[io], gen(cx + K)
    n, c, nseq = before + sum(lens) + behind, cx + 2 * cb, len(lens)
    x, w = strided(randn(g, n, c, io=io), pad), randn(g, c, K, scale=K ** -0.5)
    b = randn(g, c, scale=0.1) if bias else None
    cu = bounds(lens, before)
    slots = torch.randperm(nseq + 3, generator=g)[:nseq].to(torch.int32)
    if nseq > 2:
        slots[2] = -1
    state = randn(g, nseq + 3, c, K - 1, io=io)
    has = torch.rand(nseq, generator=g) < 0.6
    has[0] = True
    init = d64(state)[slots.clamp(min=0).long()] * (has & (slots >= 0))[:, None, None]
    want, mag, last = ref.conv(d64(x), d64(w), d64(b), cu, silu, init)
    ends = d64(state).clone()
    for i, (lo, hi) in enumerate(ref.spans(cu)):
        if hi > lo and slots[i] >= 0:
            ends[slots[i]] = last[i]
    out = tuple(torch.full((n, k), 7.0, dtype=io, device="cuda") for k in (cx, cb, cb))
    got = ssd.ssd_conv1d_varlen(x, w, b, cu, x_channels=cx, bc_channels=cb, silu=silu, conv_state=state,
                                slots=slots.cuda(), has_init=has.cuda(), out=out)
    ssd.ssd_get_device_status()
    got = torch.cat(got, 1)
    rows = slice(before, before + sum(lens))
    close(got[rows], want[rows], mag[rows], CONV_ROUNDINGS, "out")
    assert (got[:before] == 7).all() and (got[before + sum(lens):] == 7).all()
    assert torch.equal(d64(state), ends)


def test_conv_varlen_without_states_and_slots():
    g, lens = gen(3), [5, 40]
    x, w, cu = randn(g, 45, 32), randn(g, 32, 4), bounds(lens)
    want, mag, last = ref.conv(d64(x), d64(w), None, cu, True)
    close(torch.cat(ssd.ssd_conv1d_varlen(x, w, None, cu), 1), want, mag, CONV_ROUNDINGS)
    state = torch.full((2, 32, 3), float("nan"), device="cuda")  # not read: no prompt says it has one
    close(torch.cat(ssd.ssd_conv1d_varlen(x, w, None, cu, conv_state=state), 1), want, mag, CONV_ROUNDINGS)
    assert torch.equal(d64(state), last)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,cx,cb,K,pad", [(1, 64, 16, 4, 8), (5, 33, 7, 3, 1), (130, 200, 8, 4, 0), (2, 16, 0, 1, 0),
                                           (3, 5, 0, 8, 0)])
def test_conv_update(io, n, cx, cb, K, pad):
    io, g, c = IO[io], gen(n), cx + 2 * cb
    x, w, b = strided(randn(g, n, c, io=io), pad), randn(g, c, K, scale=K ** -0.5), randn(g, c, scale=0.1)
    slots = torch.randperm(n + 2, generator=g)[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
    state = randn(g, n + 2, c, K - 1, io=io)
    live = slots >= 0
    init = d64(state)[slots.clamp(min=0).long()]
    want, mag, last = ref.conv(d64(x), d64(w), d64(b), torch.arange(n + 1), True, init)
    ends = d64(state).clone()
    ends[slots[live].long()] = last[live]
    out = tuple(torch.full((n, k), 7.0, dtype=io, device="cuda") for k in (cx, cb, cb))
    got = torch.cat(ssd.ssd_conv1d_update(state, x, w, b, slots=slots.cuda(), x_channels=cx, bc_channels=cb, out=out), 1)
    ssd.ssd_get_device_status()
    close(got[live.cuda()], want[live], mag[live], CONV_ROUNDINGS)
    assert (got[~live.cuda()] == 7).all()
    assert torch.equal(d64(state), ends)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("cx,cb,K,pad,silu,bias", [(64, 16, 4, 16, True, True), (33, 7, 4, 3, True, False),
                                                   (40, 0, 3, 0, False, True), (8, 8, 2, 8, True, True),
                                                   (17, 1, 8, 1, True, True), (24, 0, 1, 0, True, True)])
def test_conv_bwd(io, lens, cx, cb, K, pad, silu, bias):
    lens, before, behind = LENS[lens]
    io, g = IO[io], gen(cx * K)
    n, c = before + sum(lens) + behind, cx + 2 * cb
    x, w = strided(randn(g, n, c, io=io), pad), randn(g, c, K, scale=K ** -0.5)
    b, cu = randn(g, c, scale=0.1) if bias else None, bounds(lens, before)
    douts = [randn(g, n, k, io=io) for k in (cx, cb, cb)]
    want = ref.conv_bwd(d64(x), d64(w), d64(b), cu, d64(torch.cat(douts, 1)), silu)
    got = ssd.ssd_conv1d_bwd(x, w, b, cu, *douts, silu=silu)
    ssd.ssd_get_device_status()
    close(got["dxbc"], *want["dxbc"], 60, "dxbc")
    close(got["dweight"], *want["dweight"], 60 + n, "dweight")
    if bias:
        close(got["dbias"], *want["dbias"], 60 + n, "dbias")
    else:
        assert got["dbias"] is None
    again = ssd.ssd_conv1d_bwd(x, w, b, cu, *douts, silu=silu)
    assert all(torch.equal(got[k], again[k]) for k in ("dxbc", "dweight"))


# --------------------------------------------------------------- selective scan

def sel_inputs(g, n, d, G, N, io, pad, D=True, z=True, bias=True, positive=False):
    """x, dt, A, B, C, then D, z, dt_bias (or None).  positive: steps ready for use."""
    A = -(torch.rand(d, N, generator=g) * 15 + 1).cuda()
    mk = lambda *s, scale=1.0: strided(randn(g, n, *s, io=io, scale=scale), pad)  # noqa: E731
    dt = mk(d, scale=0.7)
    if positive:
        dt = strided(dt.abs() * 0.1, pad)
    return (mk(d), dt, A, mk(G, N), mk(G, N)), (
        randn(g, d) if D else None, mk(d) if z else None, randn(g, d, scale=0.5) - 2.5 if bias else None)


def sel_roundings(longest, N, ins, opt, softplus=True):
    """Per step of the recurrence: the exponential (its argument is rounded twice, which
    counts as often as the argument is large, and 2^-22 of its own makes 4), the input's
    and the state's products, the step size (4: softplus); then the sum over states, the
    scan over lanes and the gate."""
    _, delta = ref.step_size(d64(ins[1]), d64(opt[2]), softplus)
    arg = float(delta.abs().max() * ins[2].abs().max()) * 1.4427 if delta.numel() else 0.0
    return longest * (6 * arg + 12) + N + 100


SEL_CASES = [(16, 1, 16, 0, True), (64, 1, 16, 8, True), (50, 2, 8, 3, True), (33, 1, 4, 0, False), (70, 1, 32, 2, True),
             (9, 3, 7, 1, True), (40, 1, 64, 4, True), (5, 1, 1, 0, True)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("d,G,N,pad,full", SEL_CASES)
def test_scan_varlen(io, lens, d, G, N, pad, full):
    lens, before, behind = LENS[lens]
    io, g = IO[io], gen(d + N)
    n, nseq = before + sum(lens) + behind, len(lens)
    ins, opt = sel_inputs(g, n, d, G, N, io, pad, full, full, full)
    cu = bounds(lens, before)
    slots = torch.randperm(nseq + 3, generator=g)[:nseq].to(torch.int32)
    if nseq > 2:
        slots[2] = -1
    state = randn(g, nseq + 3, d, N)
    has = torch.rand(nseq, generator=g) < 0.6
    has[0] = True
    init = d64(state)[slots.clamp(min=0).long()] * (has & (slots >= 0))[:, None, None]
    want, mag, end, mend, _ = ref.sel(*map(d64, ins), cu, *map(d64, opt), softplus=full, init=init)
    ends, mends = d64(state).clone(), torch.zeros_like(d64(state))
    for i, (lo, hi) in enumerate(ref.spans(cu)):
        if hi > lo and slots[i] >= 0:
            ends[slots[i]], mends[slots[i]] = end[i], mend[i]
    y = torch.full((n, d), 7.0, dtype=io, device="cuda")
    got, kept = ssd.ssd_selective_scan_varlen(*ins, cu, *opt, softplus=full, state=state, slots=slots.cuda(),
                                              has_init=has.cuda(), y=y)
    ssd.ssd_get_device_status()
    assert got is y and kept is None
    r, rows = sel_roundings(max(lens), N, ins, opt, full), slice(before, before + sum(lens))
    fits = ref.growth_fits(d64(ins[1]), d64(ins[2]), cu, d64(opt[2]), full)
    in_y, in_state = torch.ones(n, d, dtype=torch.bool), torch.ones(state.shape, dtype=torch.bool)
    for i, (lo, hi) in enumerate(ref.spans(cu)):
        in_y[lo:hi] = fits[i]
        if slots[i] >= 0:
            in_state[slots[i]] = fits[i][:, None]
    assert not full or fits.all()
    close(got[rows], want[rows], mag[rows], r, "y", in_y[rows])
    assert (got[:before] == 7).all() and (got[before + sum(lens):] == 7).all()
    close(state, ends, mends, r, "state", in_state)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_varlen_steps_as_given(io):
    """Without softplus, bias, gate and skip: steps after the softplus, as the other scans take them."""
    g = gen(21)
    ins, opt = sel_inputs(g, 300, 40, 1, 16, IO[io], 2, False, False, False, positive=True)
    cu = bounds([200, 100])
    want, mag, *_ = ref.sel(*map(d64, ins), cu, softplus=False)
    close(ssd.ssd_selective_scan_varlen(*ins, cu, softplus=False)[0], want, mag, sel_roundings(200, 16, ins, opt, False))


def test_scan_varlen_one_sequence_many_channels_and_few():
    """Both splits of a warp (by the number of blocks): the same values."""
    g = gen(11)
    for d in (8, 6000):
        ins, opt = sel_inputs(g, 300, d, 1, 4, torch.float32, 0)
        want, mag, *_ = ref.sel(*map(d64, ins), bounds([300]), *map(d64, opt))
        close(ssd.ssd_selective_scan_varlen(*ins, bounds([300]), *opt)[0], want, mag, sel_roundings(300, 4, ins, opt))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,G,N,pad,full", [(1, 64, 1, 16, 8, True), (3, 33, 1, 4, 1, False), (70, 96, 2, 8, 0, True),
                                              (5, 50, 2, 32, 2, True), (4, 9, 3, 7, 1, True), (2, 40, 1, 64, 0, True)])
def test_state_update(io, n, d, G, N, pad, full):
    io, g = IO[io], gen(n + d)
    ins, opt = sel_inputs(g, n, d, G, N, io, pad, full, full, full)
    slots = torch.randperm(n + 2, generator=g)[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
    state, live = randn(g, n + 2, d, N), slots >= 0
    want, mag, end, mend, _ = ref.sel(*map(d64, ins), torch.arange(n + 1), *map(d64, opt), softplus=full,
                                      init=d64(state)[slots.clamp(min=0).long()])
    ends, mends = d64(state).clone(), torch.zeros_like(d64(state))
    ends[slots[live].long()], mends[slots[live].long()] = end[live], mend[live]
    y = torch.full((n, d), 7.0, dtype=io, device="cuda")
    ssd.ssd_selective_state_update(state, *ins, *opt, softplus=full, slots=slots.cuda(), y=y)
    ssd.ssd_get_device_status()
    r = sel_roundings(1, N, ins, opt, full)
    close(y[live.cuda()], want[live], mag[live], r, "y")
    assert (y[~live.cuda()] == 7).all()
    close(state, ends, mends, r, "state")


# ------------------------------------------------------------------------ norms

# sum of squares and its mean (a tree of width terms: below 20 + width / 512 roundings), root,
# divide, products, the gate's sigmoid
NORM_ROUNDINGS = 80
WIDTHS = [1, 7, 64, 100, 512, 1000, 2048, 2049, 4096, 8192]


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("rows,pad,scaled,residual", [(1, 0, False, True), (5, 8, True, True), (130, 1, True, True),
                                                      (9, 0, True, False)])
def test_residual_rmsnorm(io, res, width, rows, pad, scaled, residual):
    g, io, res = gen(width), IO[io], IO[res]
    x, r0 = strided(randn(g, rows, width, io=io), pad), strided(randn(g, rows, width, io=res, scale=3.0), pad) if residual else None
    w, s = 1 + randn(g, width, scale=0.1), torch.rand(width, generator=g).cuda() if scaled else None
    want, wr, mo, mr = ref.norm_before(d64(x), d64(w), d64(r0), d64(s))
    out, r = ssd.ssd_residual_rmsnorm(x, w, r0, s)
    assert r.dtype == (res if residual else io)
    close(out, want, mo, NORM_ROUNDINGS, "out")
    close(r, wr, mr, 4, "r")
    dout, dres = randn(g, rows, width, io=io), randn(g, rows, width, io=r.dtype)
    for upstream in (dres, None):
        grads = ref.norm_before_bwd(d64(r), d64(w), d64(dout), d64(upstream), d64(x), d64(s))
        got = ssd.ssd_residual_rmsnorm_bwd(r, w, dout, upstream, x, s)
        for k, (v, m) in grads.items():
            close(got[k], v, m, NORM_ROUNDINGS + (rows if k in ("dweight", "dscale") else 0), k)
        assert ("dscale" in grads) == (got["dscale"] is not None)
    ssd.ssd_get_device_status()


def test_residual_rmsnorm_in_place():
    g = gen(5)
    x, r0, w = randn(g, 33, 512, io=torch.bfloat16), randn(g, 33, 512), 1 + randn(g, 512, scale=0.1)
    out, r = ssd.ssd_residual_rmsnorm(x, w, r0)
    kept = r0.clone()
    out2, r2 = ssd.ssd_residual_rmsnorm(x, w, kept, residual_out=kept)
    assert r2 is kept and torch.equal(r2, r) and torch.equal(out, out2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("width,G", [(1, 1), (7, 7), (100, 4), (512, 8), (1000, 1), (1000, 8), (4096, 1), (4096, 8), (8200, 2)])
@pytest.mark.parametrize("rows,pad,scaled,residual,gated", [(1, 0, False, False, True), (5, 8, True, True, True),
                                                            (130, 1, True, False, True), (9, 0, False, True, False)])
@pytest.mark.parametrize("first", [False, True])
def test_gated_rmsnorm(io, width, G, rows, pad, scaled, residual, gated, first):
    g, io = gen(width + G), IO[io]
    y, z = strided(randn(g, rows, width, io=io), pad), strided(randn(g, rows, width, io=io), pad) if gated else None
    r0 = strided(randn(g, rows, width, io=io), pad) if residual else None
    w, s = 1 + randn(g, width, scale=0.1), torch.rand(width, generator=g).cuda() if scaled else None
    want, mag = ref.norm_after(d64(y), d64(z), d64(w), d64(r0), d64(s), G, first)
    out = ssd.ssd_gated_rmsnorm(y, z, w, r0, s, ngroups=G, norm_before_gate=first)
    close(out, want, mag, NORM_ROUNDINGS, "out")
    dout = randn(g, rows, width, io=io)
    grads = ref.norm_after_bwd(d64(y), d64(z), d64(w), d64(dout), d64(s), G, first)
    got = ssd.ssd_gated_rmsnorm_bwd(y, z, w, dout, s, ngroups=G, norm_before_gate=first)
    ssd.ssd_get_device_status()
    for k, (v, m) in grads.items():
        if k == "dz" and not gated:
            assert got[k] is None
        else:
            close(got[k], v, m, NORM_ROUNDINGS + (rows if k in ("dweight", "dscale") else 0), k)
    assert ("dscale" in grads) == (got["dscale"] is not None)


def test_norm_gradients_over_many_rows():
    """More rows than the blocks take at once; repeatable to the bit."""
    g = gen(9)
    r, w, dout = randn(g, 5003, 96), 1 + randn(g, 96, scale=0.1), randn(g, 5003, 96)
    a, b = (ssd.ssd_residual_rmsnorm_bwd(r, w, dout) for _ in range(2))
    want = ref.norm_before_bwd(d64(r), d64(w), d64(dout))
    close(a["dweight"], *want["dweight"], NORM_ROUNDINGS + 5003)
    assert a["dx"] is a["dresidual"]
    assert all(torch.equal(a[k], b[k]) for k in ("dweight", "dx"))
    empty = ssd.ssd_residual_rmsnorm_bwd(r[:0], w, dout[:0])
    assert (empty["dweight"] == 0).all()


# ----------------------------------------------------- the scan's gradient

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("d,G,N,pad,full", SEL_CASES)
def test_scan_bwd(io, lens, d, G, N, pad, full):
    lens, before, behind = LENS[lens]
    io, g = IO[io], gen(d * N)
    n = before + sum(lens) + behind
    ins, opt = sel_inputs(g, n, d, G, N, io, pad, full, full, full, positive=not full)
    cu, dy = bounds(lens, before), randn(g, n, d, io=io)
    want = ref.sel_bwd(*map(d64, ins), cu, d64(dy), *map(d64, opt), softplus=full)
    _, kept = ssd.ssd_selective_scan_varlen(*ins, cu, *opt, softplus=full, return_chunk_states=True)
    got = ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, *opt, softplus=full)
    ssd.ssd_get_device_status()
    # both recurrences, then the sums: over states, channels (dB, dC), tokens (dA, dD, ddt_bias)
    r = 2 * sel_roundings(max(lens), N, ins, opt, full)
    for k, (v, m) in want.items():
        if not full and k in ("dD", "dz", "ddt_bias"):
            assert got[k] is None
        else:
            # dB and dC in bf16: each product enters its sum without its bits past tf32's
            # eleven, less than 2^-10 = 2^14 2^-24 of it, so the sum is off by less than 2^-10 M
            short = 2 ** 14 if io == torch.bfloat16 and k in ("dB", "dC") else 0
            close(got[k], v, m, r + (n if k in ("dA", "dD", "ddt_bias") else d) + short, k)
    again = ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, *opt, softplus=full)
    assert all(got[k] is None or torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("K", [2, 3, 4, 6, 8])
@pytest.mark.parametrize("cx", [16, 5])
def test_conv_sees_no_row_past_its_width(K, cx):
    """An infinite input reaches the K rows of its own sequence that have it in their
    window and no other, in both directions."""
    g, n, bad = gen(K), 200, 100
    for t0, cu in ((bad, bounds([n])), (bad, bounds([bad + 1, n - bad - 1])), (bad, bounds([bad - 1, n - bad + 1]))):
        x, w, up = randn(g, n, cx), randn(g, cx, K), randn(g, n, cx)
        x[t0] = float("inf")
        lo, hi = next((a, b) for a, b in ref.spans(cu) if a <= t0 < b)
        out = ssd.ssd_conv1d_varlen(x, w, None, cu, silu=False)[0]
        touched = torch.zeros(n, dtype=torch.bool, device="cuda")
        touched[t0:min(t0 + K, hi)] = True
        assert torch.equal(~torch.isfinite(out).all(1), touched)
        up[t0] = float("inf")
        dx = ssd.ssd_conv1d_bwd(torch.zeros_like(x), w, None, cu, up, silu=False)["dxbc"]
        touched[:] = False
        touched[max(t0 - K + 1, lo):t0 + 1] = True
        assert torch.equal(~torch.isfinite(dx).all(1), touched)
