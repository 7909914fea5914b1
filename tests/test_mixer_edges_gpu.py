"""The mixer-block operators where earlier forms of them went wrong: outputs that come back
in a dict of the caller's, sums that cancel, infinities, growing states, caches without a
state, streams and errors of other calls."""
import ctypes

import pytest
import torch

import mixer_ref as ref
import selective_state_space_22_b200 as ssd
from mixer_ref import close, d64
from parity import to_dev
from selective_state_space_22_b200 import inputs
from test_mixer_gpu import IO, NORM_ROUNDINGS, bounds, gen, randn, sel_inputs, sel_roundings

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()


# ------------------------------------------------------------- the caller's dict of outputs

def test_scaled_norm_gradient_into_the_dict_of_an_unscaled_call():
    """Without scale dx and dresidual are one tensor; with scale they differ, and a dict that
    holds them as one gets a dx of its own."""
    g, n, d = gen(81), 19, 512
    r, w, dout, up, x = randn(g, n, d), 1 + randn(g, d, scale=0.1), randn(g, n, d), randn(g, n, d), randn(g, n, d)
    s = 2 + randn(g, d, scale=0.1)
    kept = ssd.ssd_residual_rmsnorm_bwd(r, w, dout, up)
    first = kept["dresidual"]
    assert kept["dx"] is first
    want = ssd.ssd_residual_rmsnorm_bwd(r, w, dout, up, x, s)
    got = ssd.ssd_residual_rmsnorm_bwd(r, w, dout, up, x, s, out=kept)
    assert got is kept and got["dresidual"] is first and got["dx"] is not first
    assert all(torch.equal(got[k], want[k]) for k in ("dresidual", "dx", "dweight", "dscale"))
    # the same memory under two tensors, and memory that overlaps in part, are refused
    both = torch.empty(n + 1, d, device="cuda")
    for a, b in ((both[:n], both[:n]), (both[:n], both[1:])):
        with pytest.raises(ValueError, match="share memory"):
            ssd.ssd_residual_rmsnorm_bwd(r, w, dout, up, x, s, out=dict(dx=a, dresidual=b))
    with pytest.raises(ValueError, match="share memory"):  # rows that lie a row apart
        ssd.ssd_residual_rmsnorm_bwd(r, w, dout, up, out=dict(dx=both[:n], dresidual=both[1:]))
    for _ in range(2):  # without scale one tensor for both stays what it was
        again = ssd.ssd_residual_rmsnorm_bwd(r, w, dout, up, out=dict(dx=first, dresidual=first))
        assert again["dx"] is first and again["dresidual"] is first and torch.equal(first, want["dresidual"])


def test_gradients_of_absent_inputs_are_none_in_a_dict_that_held_them():
    g, n, d, N = gen(82), 21, 24, 8
    ins, (D, z, bias) = sel_inputs(g, n, d, 1, N, torch.float32, 0)
    cu, dy, w, b, nw = bounds([n]), randn(g, n, d), randn(g, d, 4), randn(g, d), 1 + randn(g, d, scale=0.1)
    _, kept = ssd.ssd_selective_scan_varlen(*ins, cu, D, z, bias, return_chunk_states=True)
    x = ins[0]
    calls = [(lambda **o: ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, D, z, bias, **o),
              lambda **o: ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, **o), ("dD", "dz", "ddt_bias")),
             (lambda **o: ssd.ssd_conv1d_bwd(x, w, b, cu, dy, **o), lambda **o: ssd.ssd_conv1d_bwd(x, w, None, cu, dy, **o), ("dbias",)),
             (lambda **o: ssd.ssd_residual_rmsnorm_bwd(x, nw, dy, None, x, nw, **o), lambda **o: ssd.ssd_residual_rmsnorm_bwd(x, nw, dy, **o),
              ("dscale",)),
             (lambda **o: ssd.ssd_gated_rmsnorm_bwd(x, z, nw, dy, nw, **o), lambda **o: ssd.ssd_gated_rmsnorm_bwd(x, None, nw, dy, **o),
              ("dz", "dscale"))]
    for full, bare, absent in calls:
        out = full()
        assert all(out[k] is not None for k in absent)
        want = bare()
        got = bare(out=out)
        assert got is out and all(got[k] is None for k in absent), absent
        assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None)
        back = full(out=out)  # and they come again where their inputs do
        assert all(torch.equal(back[k], v) for k, v in full().items())


# ------------------------------------------------------------- sums over channels

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,G,N", [(64, 1, 4), (60, 2, 8), (35, 1, 16), (128, 2, 32), (200, 1, 64), (66, 3, 7)])
@pytest.mark.parametrize("lens", [[1] * 13, [37], [5, 0, 8]])
def test_gradients_of_b_and_c_where_channels_cancel(io, d, G, N, lens):
    """Products of 13 bits, 241 * 17 = 4097, in one half of a group's channels and -64 * 64 in
    the other: every partial sum is a whole number below 2^24, so that float32 sums are exact
    in any order, and the sum is the number of pairs.  (Products cut to 11 bits sum to zero.)
    The decays are zero, so that each token stands alone; dB takes its products from x and dy
    as well."""
    n, io, per = sum(lens), IO[io], d // G
    half = (torch.arange(d) % per < per // 2).cuda()
    odd = (torch.arange(d) % per == per - 1).cuda() & (per % 2 == 1)  # without a partner: zero
    x = torch.where(half, 241.0, 64.0).expand(n, d)
    dy = torch.where(odd, 0.0, torch.where(half, 17.0, -64.0)).expand(n, d)
    one = torch.ones(n, G, N, device="cuda", dtype=io)
    A = torch.full((d, N), -1e30, device="cuda")
    ins = (x.to(io).contiguous(), torch.ones(n, d, device="cuda", dtype=io), A, one, one)
    cu = bounds(lens)
    _, kept = ssd.ssd_selective_scan_varlen(*ins, cu, softplus=False, return_chunk_states=True)
    got = ssd.ssd_selective_scan_bwd(*ins, cu, dy.to(io).contiguous(), kept, softplus=False)
    ssd.ssd_get_device_status()
    for k in ("dB", "dC"):
        assert (got[k] == per // 2).all(), (k, got[k].flatten()[:4])


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,G,N", [(40, 1, 4), (66, 2, 8), (33, 1, 16), (36, 1, 7), (70, 1, 32), (40, 2, 64)])
@pytest.mark.parametrize("lens,t0", [([5, 30], 17), ([35], 18), ([35], 34), ([6, 2, 27], 7), ([75], 42)])
def test_an_infinity_reaches_the_gradients_that_have_it_in_their_sums_and_no_other(io, d, G, N, lens, t0, full):
    """One infinite x or dy of a channel: B's and C's gradients of the other tokens, groups
    and states, and the other channels' gradients, are what the formulas say.  Decays are mild
    and every input is away from zero, so that no 0 * infinity arises in the formulas but in
    what is infinite anyway."""
    n, io, g, c0 = sum(lens), IO[io], gen(d + t0), d // 2
    mk = lambda *s: (torch.rand(n, *s, generator=g) + 0.5).to(io).cuda()  # noqa: E731
    cu, A = bounds(lens), -(torch.rand(d, N, generator=g) * 2 + 0.1).cuda()
    for where in ("x", "dy"):
        x, dt, B, C, dy = mk(d), mk(d) * 0.1, mk(G, N), mk(G, N), mk(d)
        (x if where == "x" else dy)[t0, c0] = float("inf")
        opt = (mk(d)[0].float().contiguous(), mk(d), -mk(d)[0].float() - 1) if full else (None,) * 3
        want = ref.sel_bwd(d64(x), d64(dt), d64(A), d64(B), d64(C), cu, d64(dy), *map(d64, opt), softplus=full)
        _, kept = ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu, *opt, softplus=full, return_chunk_states=True)
        got = ssd.ssd_selective_scan_bwd(x, dt, A, B, C, cu, dy, kept, *opt, softplus=full)
        ssd.ssd_get_device_status()
        r = 2 * sel_roundings(max(lens), N, (x, dt, A), opt, full) + d
        for k, (v, m) in want.items():
            if got[k] is None:
                assert not full and k in ("dD", "dz", "ddt_bias")
                continue
            assert torch.equal(torch.isfinite(d64(got[k])), torch.isfinite(v)), (where, k)
            close(got[k], v, m, r + n, k, torch.isfinite(v))


# ------------------------------------------------------------- states that grow

def grow_case(lens, d, N, g):
    """Steps below zero for 40 tokens of each sequence (states grow by 2^200 in all there)
    from states of about 2^-107, then steps above zero that take it back; before that, states
    of zero through a growth of 2^200.  No input lies near zero, so that what grows has its
    24 bits."""
    n = sum(lens)
    away = lambda *s: (torch.rand(s, generator=g) + 0.5) * (torch.randint(2, s, generator=g) * 2 - 1)  # noqa: E731
    A = -torch.linspace(0.9, 1.0, d * N).reshape(d, N)
    dt, x = torch.full((n, d), 0.01), torch.zeros(n, d)
    at = 0
    for length in lens:
        dt[at + 8:at + 48] = -200 / 1.4427 / 40        # from nothing: stays nothing
        x[at + 60] = away(d) * 2.0 ** -100
        dt[at + 80:at + 120] = -200 / 1.4427 / 40      # up to about 2^93
        dt[at + 128:at + 168] = 200 / 1.4427 / 40      # and back
        x[at + 170:at + length] = away(length - 170, d)
        at += length
    B, C = away(n, 1, N), away(n, 1, N)
    return [t.cuda() for t in (x, dt, A.contiguous(), B, C)]


@pytest.mark.parametrize("lens,d,N", [([300], 6, 4), ([200, 250], 40, 16), ([2600], 4096, 2)])
def test_states_that_grow_within_float32(lens, d, N):
    """No product of decays but a state itself has to fit a float32, wherever the sequence is cut."""
    g = gen(83)
    ins, cu = grow_case(lens, d, N, g), bounds(lens)
    state = torch.zeros(len(lens), d, N, device="cuda")
    y, kept = ssd.ssd_selective_scan_varlen(*ins, cu, softplus=False, state=state, return_chunk_states=True)
    want, mag, end, mend, _ = ref.sel(*map(d64, ins), cu, softplus=False)
    # exponents of 139 twice on the way: as rounded products over 40 tokens (3 * 139 roundings
    # of the argument and 6 per token), or as a sum of a segment's steps, here of 96 tokens at
    # most, each addition rounded
    r = 2 * (3 * 139 + 6 * 40 + 96 * 139)
    close(y, want, mag, r, "y")
    close(state, end, mend, r, "state")
    dy = torch.zeros_like(y)
    for lo, hi in ref.spans(cu):
        dy[lo + 62] = randn(g, d, scale=2.0 ** -100)  # backwards: the later growth meets no gradient, the earlier a small one
    got = ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, softplus=False)
    grads = ref.sel_bwd(*map(d64, ins), cu, d64(dy), softplus=False)
    ssd.ssd_get_device_status()
    for k in ("dx", "ddt", "dA", "dB", "dC"):
        close(got[k], *grads[k], 2 * r + d + (sum(lens) if k == "dA" else 0), k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,N", [(40, 4), (33, 16), (40, 64), (9, 7), (96, 32)])
def test_a_token_with_a_step_of_nothing_is_the_scans(io, d, N):
    """A = -infinity and a step of exactly zero: the token leaves the state as it was, as it
    does inside a prompt (and any other step forgets it)."""
    g, b = gen(84), 3
    x, B, C = (randn(g, b, *s, io=IO[io]) for s in ((d,), (1, N), (1, N)))
    dt = torch.zeros(b, d, device="cuda", dtype=IO[io])
    dt[1] = 0.5
    A = -randn(g, d, N).abs()
    A[:, 0], A[1, N - 1] = -float("inf"), -3e38
    start = randn(g, b, d, N)
    one, whole = start.clone(), start.clone()
    y = ssd.ssd_selective_state_update(one, x, dt, A, B, C, softplus=False)
    has = torch.ones(b, dtype=torch.bool, device="cuda")
    yw, _ = ssd.ssd_selective_scan_varlen(x, dt, A, B, C, bounds([1] * b), softplus=False, state=whole, has_init=has)
    ssd.ssd_get_device_status()
    assert torch.isfinite(one).all() and torch.isfinite(y).all()
    for i in (0, 2):
        assert torch.equal(one[i], start[i]) and torch.equal(whole[i], start[i])
    fresh = (dt[1].double() * x[1].double())[:, None] * B[1, 0].double()
    assert ((one[1, :, 0].double() - fresh[:, 0]).abs() <= 2 * 2.0 ** -24 * fresh[:, 0].abs()).all()
    # per state and token: exponential (argument rounded, 2^-22 of its own), three products
    tol = 40 * 2.0 ** -24 * (start.abs() + fresh.float().abs() + 1)
    assert ((one - whole).abs() <= tol).all()


# ------------------------------------------------------------- caches without a state

def test_conv_of_one_tap_has_no_state_to_find():
    """Width 1: the C call takes no cache, the Python call one of no elements, of any number of
    slots; a negative slot still skips its row."""
    g, b, d = gen(85), 5, 12
    x, w, cb = randn(g, b, d), randn(g, d, 1), randn(g, d)
    want, mag, _ = ref.conv(d64(x), d64(w), d64(cb), torch.arange(b + 1), True)
    out = torch.full((b, d), 7.0, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    lib = ssd.load_library()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.ssd_conv1d_update(None, None, p(x), d, p(w), p(cb), p(out), None, None, 0, b, 0, d, 0, 1, 1, stream) == ssd.SSD_OK
    ssd.ssd_get_device_status()
    close(out, want, mag, 40)
    for nslots in (0, 2, b):
        cache = torch.empty(nslots, d, 0, device="cuda")
        close(ssd.ssd_conv1d_varlen(x, w, cb, bounds([2, 3]), conv_state=cache)[0], want, mag, 40)
        got = ssd.ssd_conv1d_update(cache, x, w, cb)[0]
        ssd.ssd_get_device_status()
        close(got, want, mag, 40)
    out.fill_(7)
    slots = torch.tensor([4, -1, 0, 9, 4], dtype=torch.int32).cuda()
    ssd.ssd_conv1d_update(torch.empty(0, d, 0, device="cuda"), x, w, cb, slots=slots, out=(out, out[:, :0].contiguous(), out[:, :0].contiguous()))
    ssd.ssd_get_device_status()
    live = slots.cpu() >= 0
    close(out[live.cuda()], want[live], mag[live], 40)
    assert (out[1] == 7).all()


def test_a_cache_of_no_slots_is_no_missing_cache():
    """Sequences have no state to find in a cache of no slots: refused where the sequence's
    number is its slot, reported where `slots` names one; padding entries are skipped."""
    g, n, d, N = gen(86), 10, 16, 4
    (x, dt, A, B, C), _ = sel_inputs(g, n, d, 1, N, torch.float32, 0)
    cu, w = bounds([4, 6]), randn(g, d, 4)
    state, conv_state = torch.empty(0, d, N, device="cuda"), torch.empty(0, d, 3, device="cuda")
    calls = [lambda s: ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu, state=state, slots=s)[0],
             lambda s: ssd.ssd_selective_state_update(state, x[:2], dt[:2], A, B[:2], C[:2], slots=s),
             lambda s: ssd.ssd_conv1d_varlen(x, w, None, cu, conv_state=conv_state, slots=s)[0],
             lambda s: ssd.ssd_conv1d_update(conv_state, x[:2], w, slots=s)[0]]
    for call in calls:
        with pytest.raises(ssd.SSDError, match="0 states for 2 sequences"):
            call(None)
        call(torch.tensor([0, -1], dtype=torch.int32).cuda())
        with pytest.raises(ssd.SSDError) as e:
            ssd.ssd_get_device_status()
        assert e.value.status == ssd.SSD_ERR_INVALID_ARG
        call(torch.tensor([-1, -1], dtype=torch.int32).cuda())
        ssd.ssd_get_device_status()
    none = torch.tensor([-1, -1], dtype=torch.int32).cuda()
    assert torch.equal(calls[0](none), ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu)[0])
    assert torch.equal(calls[2](none), ssd.ssd_conv1d_varlen(x, w, None, cu)[0])
    ssd.ssd_get_device_status()


# ------------------------------------------------------------- errors of other calls

def test_bad_bounds_do_not_hide_a_timeout():
    """A wait that gave up invalidates a whole call, so it is reported first, whatever bounds
    or slots were refused before it; the refusal is reported by the next status call."""
    shape = inputs.ScanShape("stall", 2, 2048, 8, 64, 1, 128, 128, "bf16", init_state=True, seed=31)
    scan = to_dev(inputs.scan_inputs(shape))
    g = gen(87)
    x, w = randn(g, 10, 16), randn(g, 16, 4)
    bad = torch.tensor([0, 99], dtype=torch.int32).cuda()
    lib = ssd.load_library()
    ssd.ssd_get_device_status()
    for first in (True, False):
        try:
            if first:
                ssd.ssd_conv1d_varlen(x, w, None, bad)
            assert lib.ssd_debug_inject_stall(1, 10_000_000) == ssd.SSD_OK
            ssd.ssd_scan_fwd(scan["x"], scan["dt"], scan["A"], scan["B"], scan["C"], scan["D"], scan["init_state"], chunk_size=128)
            torch.cuda.synchronize()
        finally:
            lib.ssd_debug_inject_stall(0, 0)
        if not first:
            ssd.ssd_conv1d_varlen(x, w, None, bad)
        for status in (ssd.SSD_ERR_TIMEOUT, ssd.SSD_ERR_INVALID_ARG):
            with pytest.raises(ssd.SSDError) as e:
                ssd.ssd_get_device_status()
            assert e.value.status == status
        ssd.ssd_get_device_status()


def test_no_memory_is_torchs_error():
    """Kept states for 2^24 empty prompts of 64 channels and states (275 GB) cannot be had:
    the allocator's own error, as from any other call, and the next call runs."""
    g, d, N = gen(88), 64, 64
    (x, dt, A, B, C), _ = sel_inputs(g, 3, d, 1, N, torch.bfloat16, 0)
    cu = torch.zeros((1 << 24) + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        ssd.ssd_selective_scan_varlen(x, dt, A, B, C, cu, return_chunk_states=True)
    del cu
    y, kept = ssd.ssd_selective_scan_varlen(x, dt, A, B, C, bounds([3]), return_chunk_states=True)
    ssd.ssd_get_device_status()
    assert kept.shape == (1, N, d) and torch.isfinite(y).all()
