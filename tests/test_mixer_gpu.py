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


# ---------------------------------------------------- together, as they are used

def test_prompt_then_tokens_is_the_whole_sequence():
    """A Mamba-1 mixer as serving runs it: prompts into slots (conv, scan), then a token
    at a time, against one run over the whole sequences."""
    g, d, N, K = gen(31), 48, 16, 4
    lens, more, nslots = [37, 1, 200], 5, 6
    whole = [n + more for n in lens]
    n = sum(whole)
    xz = randn(g, n, 2 * d, io=torch.bfloat16)
    proj = randn(g, n, 8 + 2 * N, io=torch.bfloat16)  # the x projection's output: dt rank, B, C
    dt = randn(g, n, d, io=torch.bfloat16, scale=0.7)
    w, b, A = randn(g, d, K, scale=0.5), randn(g, d, scale=0.1), -(torch.rand(d, N, generator=g) * 15 + 1).cuda()
    D, bias, norm = randn(g, d), randn(g, d, scale=0.5) - 2.5, 1 + randn(g, d, scale=0.1)
    B, C = proj[:, 8:8 + N].unflatten(1, (1, N)), proj[:, 8 + N:].unflatten(1, (1, N))

    def mixer(rows, cu=None, states=None, slots=None):
        conv_state, state = states
        args = dict(slots=slots)
        xin, z = xz[rows, :d], xz[rows, d:]
        if cu is None:
            x = ssd.ssd_conv1d_update(conv_state, xin, w, b, **args)[0]
            y = ssd.ssd_selective_state_update(state, x, dt[rows], A, B[rows], C[rows], D, z, bias, **args)
        else:
            x = ssd.ssd_conv1d_varlen(xin, w, b, cu, conv_state=conv_state, **args)[0]
            y, _ = ssd.ssd_selective_scan_varlen(x, dt[rows], A, B[rows], C[rows], cu, D, z, bias, state=state, **args)
        return ssd.ssd_gated_rmsnorm(y, None, norm)

    fresh = lambda: (torch.full((nslots, d, K - 1), float("nan"), dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                     torch.full((nslots, d, N), float("nan"), device="cuda"))
    all_rows = slice(0, n)
    whole_states = fresh()
    want = mixer(all_rows, bounds(whole), whole_states, torch.arange(3, dtype=torch.int32, device="cuda"))
    first = torch.tensor([0] + whole).cumsum(0)
    prompt = torch.cat([torch.arange(first[i], first[i] + lens[i]) for i in range(3)]).cuda()
    states, slots = fresh(), torch.tensor([4, 0, 3], dtype=torch.int32, device="cuda")
    got = torch.empty_like(want)
    got[prompt] = mixer(prompt, bounds(lens), states, slots)
    for step in range(more):
        rows = torch.tensor([int(first[i]) + lens[i] + step for i in range(3)], device="cuda")
        got[rows] = mixer(rows, None, states, slots)
    ssd.ssd_get_device_status()
    # the same float32 recurrence cut at other places; then two bf16 roundings (y and the norm)
    # and what the first one does to the second
    scale = want.float().abs().amax()
    assert (got.float() - want.float()).abs().max() <= 4 * 2.0 ** -8 * scale
    assert (got == want).float().mean() > 0.9
    for a, b in zip(states, whole_states):
        assert torch.allclose(a[slots.long()].float(), b[:3].float(), rtol=1e-5, atol=1e-5)


def test_training_chain_against_differences():
    """norm before -> conv -> scan -> norm after, packed, float32: the gradients chained by
    hand against central differences of the chained forwards."""
    g, d, N, lens = gen(41), 24, 8, [50, 1, 30]
    n, cu = sum(lens), bounds(lens)
    p = dict(r=randn(g, n, d), w0=1 + randn(g, d, scale=0.1), w=randn(g, d, 4, scale=0.5), b=randn(g, d, scale=0.1),
             dt=randn(g, n, d, scale=0.7), A=-(torch.rand(d, N, generator=g) * 7 + 1).cuda(), B=randn(g, n, 1, N), C=randn(g, n, 1, N),
             D=randn(g, d), z=randn(g, n, d), bias=randn(g, d, scale=0.5) - 2, w1=1 + randn(g, d, scale=0.1))
    up = randn(g, n, d)

    def forward(r, w0, w, b, dt, A, B, C, D, z, bias, w1):
        h, res = ssd.ssd_residual_rmsnorm(r, w0)
        x = ssd.ssd_conv1d_varlen(h, w, b, cu)[0]
        y, kept = ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu, D, z, bias, return_chunk_states=True)
        return ssd.ssd_gated_rmsnorm(y, z, w1), (h, res, x, y, kept)

    _, (h, res, x, y, kept) = forward(**p)
    ga = ssd.ssd_gated_rmsnorm_bwd(y, p["z"], p["w1"], up)
    gs = ssd.ssd_selective_scan_bwd(x, p["dt"], p["A"], p["B"], p["C"], cu, ga["dy"], kept, p["D"], p["z"], p["bias"])
    gc = ssd.ssd_conv1d_bwd(h, p["w"], p["b"], cu, gs["dx"])
    gb = ssd.ssd_residual_rmsnorm_bwd(res, p["w0"], gc["dxbc"])
    grads = dict(r=gb["dx"], w0=gb["dweight"], w=gc["dweight"], b=gc["dbias"], dt=gs["ddt"], A=gs["dA"], B=gs["dB"], C=gs["dC"],
                 D=gs["dD"], z=gs["dz"] + ga["dz"], bias=gs["ddt_bias"], w1=ga["dweight"])
    loss = lambda q: (forward(**q)[0].double() * up.double()).sum().item()  # noqa: E731
    eps = 2.0 ** -7  # the difference's own error: eps^2 of a third derivative, and 2^-24 sum |out up| / eps
    noise = (forward(**p)[0].double() * up.double()).abs().sum().item() * 2.0 ** -20 / eps
    for k, v in p.items():
        v_dir = torch.randn(v.shape, generator=g).cuda() * (0.1 if k in ("A", "dt", "bias") else 1.0) / v.numel() ** 0.5
        slope = (grads[k].double() * v_dir.double()).sum().item()
        diff = (loss(dict(p, **{k: v + eps * v_dir})) - loss(dict(p, **{k: v - eps * v_dir}))) / (2 * eps)
        assert abs(diff - slope) <= 1e-2 * abs(slope) + noise + 1e-3, (k, diff, slope)


def test_bad_bounds_and_slots_are_reported_and_harmless():
    """Bounds that leave the tensor, slots out of range or named twice: nothing outside is
    touched, the rest is served, and the status says so once."""
    g, d, N, n = gen(51), 40, 16, 60
    ins, opt = sel_inputs(g, n, d, 1, N, torch.float32, 0)
    w = randn(g, d, 4)

    def reported():
        with pytest.raises(ssd.SSDError) as e:
            ssd.ssd_get_device_status()
        assert e.value.status == ssd.SSD_ERR_INVALID_ARG
        ssd.ssd_get_device_status()  # cleared

    good = ssd.ssd_selective_scan_varlen(*ins, bounds([20]), *opt)[0][:20]
    for cu in ([0, 20, 70], [-5, 20, 40], [0, 20, 10], [20, 0, 20], [0, 20, 2 ** 31 - 1], [0, 20, -2 ** 31]):
        cu = torch.tensor(cu, dtype=torch.int32).cuda()
        y = torch.full((n, d), 7.0, device="cuda")
        _, kept = ssd.ssd_selective_scan_varlen(*ins, cu, *opt, y=y, return_chunk_states=True)
        if cu[0] == 0 and cu[1] == 20:
            assert torch.equal(y[:20], good)
        reported()
        ssd.ssd_selective_scan_bwd(*ins, cu, torch.ones_like(y), kept, *opt)
        reported()
        for call in (lambda: ssd.ssd_conv1d_varlen(ins[0], w, None, cu), lambda: ssd.ssd_conv1d_bwd(ins[0], w, None, cu, ins[0])):
            call()
            reported()
    state, conv_state = torch.zeros(3, d, N, device="cuda"), torch.zeros(3, d, 3, device="cuda")
    cu, lens3 = bounds([20, 20, 20]), 3
    for slots in ([1, 3, 0], [1, 1, 0], [2, 0, 2 ** 31 - 1]):
        s = torch.tensor(slots, dtype=torch.int32).cuda()
        served = [v for v in dict.fromkeys(slots) if v < 3]
        for t in (state, conv_state):
            t.fill_(0.25)
        ssd.ssd_selective_scan_varlen(*ins, cu, *opt, state=state, slots=s)
        reported()
        ssd.ssd_conv1d_varlen(ins[0], w, None, cu, conv_state=conv_state, slots=s)
        reported()
        for t in (state, conv_state):
            for v in range(3):
                assert (t[v] == 0.25).all().item() == (v not in served), (slots, v)
        t3 = [t[:lens3] for t in ins[:2]] + [ins[2]] + [t[:lens3] for t in ins[3:]]
        o3 = (opt[0], opt[1][:lens3], opt[2])
        for t in (state, conv_state):
            t.fill_(0.25)
        y = torch.full((lens3, d), 7.0, device="cuda")
        ssd.ssd_selective_state_update(state, *t3, *o3, slots=s, y=y)
        reported()
        x = torch.full((lens3, d), 7.0, device="cuda")
        ssd.ssd_conv1d_update(conv_state, ins[0][:lens3], w, slots=s, out=(x, x[:, :0].contiguous(), x[:, :0].contiguous()))
        reported()
        for t in (state, conv_state):
            for v in range(3):
                assert (t[v] == 0.25).all().item() == (v not in served), (slots, v)
        skipped = [i for i in range(3) if slots[i] >= 3 or slots[i] in slots[:i]]
        for i in range(3):
            assert (y[i] == 7).all().item() == (i in skipped) and (x[i] == 7).all().item() == (i in skipped)


def test_on_streams_and_in_graphs():
    """Two streams at once and two captured graphs (each with its own scratch) give the
    bits of plain calls; a graph sees the inputs of its replay."""
    g, d, N, lens = gen(61), 96, 16, [3000, 200]  # few channels, long: cut into segments, with scratch
    n, cu = sum(lens), bounds(lens)
    sets = [sel_inputs(g, n, d, 1, N, torch.bfloat16, 0) for _ in range(2)]
    dy = randn(g, n, d, io=torch.bfloat16)

    def step(ins, opt, **kw):
        y, kept = ssd.ssd_selective_scan_varlen(*ins, cu, *opt, return_chunk_states=True, **kw)
        return [y] + list(ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, *opt, **kw).values())

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [step(*s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, v in zip(want, got) for a, b in zip(w, v))
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*s))
        graphs.append(graph)
    for order in ((0, 1), (1, 0)):
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, v in zip(want, outs) for a, b in zip(w, v))
    sets[0][0][0].copy_(sets[1][0][0])  # another x
    again = step(*sets[0])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, outs[0]))
    ssd.ssd_get_device_status()


def test_given_outputs_are_used_and_checked():
    g, n, d = gen(71), 9, 32
    x, w = randn(g, n, d), 1 + randn(g, d, scale=0.1)
    out, res = torch.empty_like(x), torch.empty_like(x)
    a, b = ssd.ssd_residual_rmsnorm(x, w, x, out=out, residual_out=res)
    assert a is out and b is res
    grads = dict(dresidual=torch.empty_like(x), dweight=torch.empty_like(w))
    got = ssd.ssd_residual_rmsnorm_bwd(res, w, x, out=grads)
    assert got is grads and got["dx"] is grads["dresidual"]
    for bad in (lambda: ssd.ssd_residual_rmsnorm(x, w, out=out[:, :16]), lambda: ssd.ssd_residual_rmsnorm(x, w.half()),
                lambda: ssd.ssd_residual_rmsnorm(x.half(), w), lambda: ssd.ssd_residual_rmsnorm(x.T, w), lambda: ssd.ssd_residual_rmsnorm(x, w, x.cpu()),
                lambda: ssd.ssd_residual_rmsnorm(x, None), lambda: ssd.ssd_residual_rmsnorm(x[0], w), lambda: ssd.ssd_gated_rmsnorm(x, x, w[:5]),
                lambda: ssd.ssd_residual_rmsnorm_bwd(x, w, x, scale=w), lambda: ssd.ssd_conv1d_varlen(x, w[:, None], None, bounds([n]).long()),
                lambda: ssd.ssd_conv1d_varlen(x, w[:, None], None, bounds([n]), x_channels=5), lambda: ssd.ssd_conv1d_varlen(x[:, ::2], w[::2, None], None, bounds([n])),
                lambda: ssd.ssd_conv1d_varlen(x.expand(n, d), w[:, None], None, bounds([n]), out=(out,))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssd.ssd_gated_rmsnorm(x, x, w, ngroups=3), lambda: ssd.ssd_gated_rmsnorm(x, x, w, eps=-1.0),
                lambda: ssd.ssd_residual_rmsnorm(x, torch.ones(d + 1, device="cuda")[1:])):
        with pytest.raises(ssd.SSDError):
            bad()
    empty = x[:0]
    assert ssd.ssd_residual_rmsnorm(empty, w)[0].shape == (0, d) and ssd.ssd_gated_rmsnorm(empty, empty, w).shape == (0, d)
    assert ssd.ssd_conv1d_varlen(empty, w[:, None].contiguous(), None, bounds([]))[0].shape == (0, d)
    none = ssd.ssd_conv1d_bwd(empty, w[:, None].contiguous(), None, bounds([]), empty)
    assert (none["dweight"] == 0).all()


def test_gradients_into_given_tensors_and_in_place():
    """A dx that the caller gives is filled even where it equals dresidual; dresidual may be
    the upstream one, and the gated norm's result its residual."""
    g, n, d = gen(72), 37, 512
    x, w, dout, up = randn(g, n, d), 1 + randn(g, d, scale=0.1), randn(g, n, d), randn(g, n, d)
    want = ssd.ssd_residual_rmsnorm_bwd(x, w, dout, up)
    dx = torch.full_like(x, 7.0)
    got = ssd.ssd_residual_rmsnorm_bwd(x, w, dout, up, out=dict(dx=dx))
    assert got["dx"] is dx and torch.equal(dx, want["dx"]) and torch.equal(got["dresidual"], want["dresidual"])
    again = ssd.ssd_residual_rmsnorm_bwd(x, w, dout, up, out=want)  # the dict of an earlier call
    assert again is want and torch.equal(want["dx"], dx)
    here = up.clone()
    got = ssd.ssd_residual_rmsnorm_bwd(x, w, dout, here, out=dict(dresidual=here))
    assert got["dresidual"] is here and torch.equal(here, dx) and torch.equal(got["dweight"], want["dweight"])
    res = randn(g, n, d)
    plain = ssd.ssd_gated_rmsnorm(x, dout, w, res, ngroups=2)
    assert ssd.ssd_gated_rmsnorm(x, dout, w, res, ngroups=2, out=res) is res and torch.equal(res, plain)


def test_tokens_and_norms_in_graphs():
    """A captured step of single tokens, replayed, moves the states on as plain calls do; a
    captured training step of the conv and the norms gives the bits of plain calls, on two
    streams and replayed while plain calls run."""
    g, b, d, N, K = gen(62), 5, 64, 16, 4
    ct = d + 2 * N
    w, cb, A, nw = randn(g, ct, K), randn(g, ct), -randn(g, d, N).abs(), 1 + randn(g, d, scale=0.1)
    slots = torch.tensor([3, 0, -1, 5, 1], dtype=torch.int32).cuda()
    tokens = [(randn(g, b, ct, io=torch.bfloat16), randn(g, b, d, io=torch.bfloat16), randn(g, b, d, io=torch.bfloat16)) for _ in range(6)]

    def states():
        return torch.zeros(6, ct, K - 1, device="cuda", dtype=torch.bfloat16), torch.zeros(6, d, N, device="cuda")

    def token(xbc, dt, z, conv_state, state):
        x, B, C = ssd.ssd_conv1d_update(conv_state, xbc, w, cb, slots=slots, x_channels=d, bc_channels=N)
        y = ssd.ssd_selective_state_update(state, x, dt, A, B.view(b, 1, N), C.view(b, 1, N), z=z, slots=slots)
        return ssd.ssd_gated_rmsnorm(y, z, nw)

    keep = [i for i in range(b) if i != 2]  # the skipped row's result is not written
    plain = states()
    want = [token(*t, *plain)[keep] for t in tokens]
    mine, held = states(), [t.clone() for t in tokens[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(*held, *mine)
    for t, r in zip(tokens, want):
        for a, v in zip(held, t):
            a.copy_(v)
        graph.replay()
        assert torch.equal(out[keep], r)
    assert all(torch.equal(a, v) for a, v in zip(mine, plain))

    cu, n = bounds([700, 1, 0, 323]), 1024
    xbc, z, dy, r0 = randn(g, n, ct), randn(g, n, d), randn(g, n, d), randn(g, n, d)
    dB = randn(g, n, N)

    def step(**kw):
        x, B, C = ssd.ssd_conv1d_varlen(xbc, w, cb, cu, x_channels=d, bc_channels=N, **kw)
        h, r = ssd.ssd_residual_rmsnorm(x, nw, r0, nw, **kw)
        o = ssd.ssd_gated_rmsnorm(h, z, nw, **kw)
        go = ssd.ssd_gated_rmsnorm_bwd(h, z, nw, dy, **kw)
        gr = ssd.ssd_residual_rmsnorm_bwd(r, nw, go["dy"], None, x, nw, **kw)
        gc = ssd.ssd_conv1d_bwd(xbc, w, cb, cu, gr["dx"], dB, dB, **kw)
        return [x, B, C, h, r, o] + [v for q in (go, gr, gc) for v in q.values() if v is not None]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [step(stream=st) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, v) for q in got for a, v in zip(want, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        got = step(stream=streams[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, v) and torch.equal(a, u) for a, v, u in zip(want, got, outs))
    ssd.ssd_get_device_status()


def test_offsets_past_32_bits():
    """Rows and state slots that lie past 2^31 elements give the bits of small copies."""
    g, d, N, rows = gen(63), 256, 64, 18
    ld = (1 << 27) + 64
    big = torch.empty(rows, ld, device="cuda", dtype=torch.bfloat16)
    assert (rows - 1) * ld > 1 << 31
    part = big[:, :3 * d + 2 * N]
    part.copy_(randn(g, rows, 3 * d + 2 * N))
    small = part.contiguous()

    def cut(t):
        return t[:, :d], t[:, d:2 * d], t[:, 2 * d:3 * d], t[:, 3 * d:3 * d + N].view(rows, 1, N), t[:, 3 * d + N:].view(rows, 1, N)

    A, w = -randn(g, d, N).abs(), randn(g, d, 4)
    nw, cu, slots = 1 + randn(g, d, scale=0.1), bounds([7, rows - 7]), (1 << 17) + 4
    state, few = torch.empty(slots, d, N, device="cuda"), torch.zeros(3, d, N, device="cuda")
    assert (slots - 3) * d * N > 1 << 31
    state[-3:].zero_()
    far, near = torch.tensor([slots - 1, slots - 3], dtype=torch.int32).cuda(), torch.tensor([2, 0], dtype=torch.int32).cuda()
    dy = randn(g, rows, d, io=torch.bfloat16)
    got = []
    for t, st, sl in ((part, state, far), (small, few, near)):
        x, dt, z, B, C = cut(t)
        y, kept = ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu, z=z, state=st, slots=sl, return_chunk_states=True)
        grads = ssd.ssd_selective_scan_bwd(x, dt, A, B, C, cu, dy, kept, z=z)
        first = [v[:2] for v in (x, dt, B, C, z)]
        tok = ssd.ssd_selective_state_update(st, first[0], first[1], A, first[2], first[3], z=first[4], slots=sl)
        conv = ssd.ssd_conv1d_varlen(x, w, None, cu)[0]
        gc = ssd.ssd_conv1d_bwd(x, w, None, cu, dy)
        norm, r = ssd.ssd_residual_rmsnorm(x, nw, z)
        gn = ssd.ssd_gated_rmsnorm_bwd(x, z, nw, dy)
        gr = ssd.ssd_residual_rmsnorm_bwd(x, nw, dy)
        got.append([y, tok, conv, norm, r, ssd.ssd_gated_rmsnorm(x, z, nw), st[-3:]]
                   + [v for q in (grads, gc, gn, gr) for v in q.values() if v is not None])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    ssd.ssd_get_device_status()


@pytest.mark.parametrize("lens", [[5], [3, 12, 1], [700]])
@pytest.mark.parametrize("N", [4, 16, 64])
def test_states_that_forget_everything(lens, N):
    """A = -infinity (and one whose product with a step leaves float32): such a state holds its
    last input alone, whatever the sequence's length, and hands no gradient back."""
    g, n, d = gen(73), sum(lens), 34
    (x, dt, A, B, C), opt = sel_inputs(g, n, d, 1, N, torch.float32, 0)
    A[:, 1], A[3, 2] = -float("inf"), -3e38
    cu, state = bounds(lens), torch.zeros(len(lens), d, N, device="cuda")
    y, kept = ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu, *opt, state=state, return_chunk_states=True)
    grads = ssd.ssd_selective_scan_bwd(x, dt, A, B, C, cu, torch.ones_like(y), kept, *opt)
    assert all(torch.isfinite(v).all() for v in [y, state, *grads.values()])
    assert (grads["dA"][:, 1] == 0).all() and grads["dA"][3, 2] == 0
    last = cu[1:].long() - 1
    delta = torch.nn.functional.softplus((dt[last] + opt[2]).double())
    want = delta * x[last].double() * B[last, 0, 1:2].double()
    # softplus and its approximate exponential (as in the scans' other tests: 64 roundings), two products
    assert ((state[:, :, 1].double() - want).abs() <= 66 * 2.0 ** -24 * want.abs()).all()
    mild = A.clamp(min=-1e4)  # exp(-1e4 step) is zero in float32 too, for steps above 0.011
    if (torch.nn.functional.softplus(dt + opt[2]) > 0.011).all():
        assert torch.equal(y, ssd.ssd_selective_scan_varlen(x, dt, mild, B, C, cu, *opt)[0])
    ssd.ssd_get_device_status()
