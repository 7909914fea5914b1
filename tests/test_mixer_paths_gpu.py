"""The mixer-block operators on the paths that large calls take: scans whose sequences are
not cut and scans cut into long segments, norms of many rows and of channel pairs.  Each test
first makes sure, by the size of the workspace, that its path is the one meant."""
import pytest
import torch

import mixer_ref as ref
import selective_state_space_22_b200 as ssd
from mixer_bounds import Scan, within
from mixer_ref import close, d64
from test_mixer_gpu import IO, NORM_ROUNDINGS, bounds, gen, randn, sel_inputs, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ssd.load_library()


def fwd_seg(n, nseq, d, N):
    """Tokens of the forward's segments, 0 where sequences are not cut: a cut call has
    d (N + 1) floats for each of n / seg + nseq segments."""
    size = ssd.load_library().ssd_selective_scan_workspace_size(n, nseq, d, N)
    slots = size // (4 * d * (N + 1))
    return slots and {n // s + nseq: s for s in range(n + 1, 0, -1)}[slots]


def bwd_seg(n, nseq, d, G, N):
    """The same of the gradient: per segment d (2 N + 3) floats where sequences are cut, else
    d (N + 2) per sequence, beside the channel tiles' sums of dB and dC."""
    split = 1 if N <= 8 else 2 if N <= 16 else 4
    tiles = (d // G + 256 // split - 1) // (256 // split)
    size = ssd.load_library().ssd_selective_scan_bwd_workspace_size(n, nseq, d, G, N) // 4 - G * tiles * n * 2 * N
    if size == nseq * d * (N + 2):
        return 0
    slots = size // (d * (2 * N + 3))
    assert slots * d * (2 * N + 3) == size
    return {n // s + nseq: s for s in range(n + 1, 0, -1)}[slots]


def test_the_segments_are_found_by_the_workspace():
    """fwd_seg and bwd_seg give a length with the same number of segments as the one chosen."""
    assert fwd_seg(300, 2, 64, 16) and bwd_seg(300, 2, 64, 1, 16)
    assert fwd_seg(64 * 512, 64, 1024, 16) == 0 and bwd_seg(64 * 512, 64, 1024, 1, 16) == 0


def run_scan(ins, opt, cu, softplus, io, seg, bseg, g, before=0):
    """Forward with states and slots, then forward and gradient without; all against the bounds."""
    x, nseq = ins[0], cu.numel() - 1
    n, d = x.shape
    N = ins[2].shape[1]
    slots = torch.randperm(nseq + 3, generator=g)[:nseq].to(torch.int32)
    slots[2::7] = -1
    has = torch.rand(nseq, generator=g) < 0.6
    has[0] = True
    state = randn(g, nseq + 3, d, N)
    init = d64(state)[slots.clamp(min=0).long()] * (has & (slots >= 0))[:, None, None]
    plain = [*map(d64, ins), cu.cpu(), *map(d64, opt)]
    want = Scan(*plain, softplus=softplus, init=init, seg=seg)
    ends, ee = d64(state).clone(), torch.zeros_like(d64(state))
    for i, (lo, hi) in enumerate(ref.spans(cu)):
        if hi > lo and slots[i] >= 0:
            ends[slots[i]], ee[slots[i]] = want.end[i], want.eend[i]
    y = torch.full((n, d), 7.0, dtype=io, device="cuda")
    ssd.ssd_selective_scan_varlen(*ins, cu, *opt, softplus=softplus, state=state, slots=slots.cuda(), has_init=has.cuda(), y=y)
    ssd.ssd_get_device_status()
    rows = slice(int(cu[0]), int(cu[-1]))
    within(y[rows], (want.y[rows], want.ey[rows]), "y")
    assert (y[:rows.start] == 7).all() and (y[rows.stop:] == 7).all()
    within(state, (ends, ee), "state")
    want = Scan(*plain, softplus=softplus, seg=max(seg, bseg))
    y, kept = ssd.ssd_selective_scan_varlen(*ins, cu, *opt, softplus=softplus, return_chunk_states=True)
    within(y[rows], (want.y[rows], want.ey[rows]), "y")
    for lo, hi in ref.spans(cu)[:40]:  # the states before every 8th token
        i = ref.spans(cu).index((lo, hi))
        for k in range(8, hi - lo, 8):
            within(kept[lo // 8 + i + k // 8].T, (want.h[lo + k - 1], want.eh[lo + k - 1]), "kept")
    dy = randn(g, n, d, io=io)
    grads = want.bwd(d64(dy))
    got = ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, *opt, softplus=softplus)
    ssd.ssd_get_device_status()
    for k, v in grads.items():
        if got[k] is not None:
            within(got[k], v, k)
    assert all(got[k] is not None for k in ("dx", "ddt", "dA", "dB", "dC"))
    again = ssd.ssd_selective_scan_bwd(*ins, cu, dy, kept, *opt, softplus=softplus)
    assert all(got[k] is None or torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,G,N,pad,full,nseq", [(256, 1, 16, 8, True, 160), (250, 2, 7, 3, True, 330), (96, 1, 64, 0, True, 400),
                                                 (33, 1, 32, 1, False, 600), (129, 3, 4, 2, True, 500), (64, 1, 16, 0, False, 600)])
def test_scan_of_sequences_that_are_not_cut(io, d, G, N, pad, full, nseq):
    g = gen(d + N)
    lens = [(0, 1, 2, 3, 4, 5, 8, 9)[int(k)] for k in torch.randint(8, (nseq,), generator=g)]
    lens[3], lens[nseq // 2], lens[-2] = 70, 33, 17
    before, behind = 3, 5
    n = before + sum(lens) + behind
    assert fwd_seg(n, nseq, d, N) == 0 and bwd_seg(n, nseq, d, G, N) == 0
    ins, opt = sel_inputs(g, n, d, G, N, IO[io], pad, full, full, full, positive=not full)
    run_scan(ins, opt, bounds(lens, before), full, IO[io], 0, 0, g)


@pytest.mark.parametrize("io,lens,d,G,N,seg", [("bf16", [1650, 49, 1], 2048, 1, 16, 48), ("f32", [1650, 49, 1], 4094, 2, 3, 48),
                                               ("f32", [2300, 0, 499, 1], 16384, 1, 1, 304), ("bf16", [2300, 0, 499, 1], 8191, 1, 1, 160)])
def test_scan_cut_into_long_segments(io, lens, d, G, N, seg):
    g, n, nseq = gen(N), sum(lens), len(lens)
    for got in (fwd_seg(n, nseq, d, N), bwd_seg(n, nseq, d, G, N)):
        assert n // got == n // seg, got
    ins, opt = sel_inputs(g, n, d, G, N, IO[io], 0)
    run_scan(ins, opt, bounds(lens), True, IO[io], seg, seg, g)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5], [3, 12, 1], [700], [1, 0, 2] * 200])
@pytest.mark.parametrize("d,N", [(34, 4), (64, 16), (48, 64)])
def test_values_beside_states_that_forget_everything(io, lens, d, N):
    """Every step is 0.02 or more, so that a rate of -infinity (or one that leaves float32
    with the step) and one of -1e5 decay a state to zero alike, in 64 bits too."""
    g, n = gen(74), sum(lens)
    (x, dt, A, B, C), (D, z, _) = sel_inputs(g, n, d, 1, N, IO[io], 0)
    dt = (dt.float().abs() * 0.1 + 0.02).to(IO[io])
    mild = A.clone()
    A[:, 1], mild[:, 1] = -float("inf"), -1e5
    A[3, 2], mild[3, 2] = -3e38, -1e5
    cu, state = bounds(lens), torch.zeros(len(lens), d, N, device="cuda")
    args = (x, dt, A, B, C, cu, D, z)
    y, kept = ssd.ssd_selective_scan_varlen(*args, softplus=False, state=state, return_chunk_states=True)
    want = Scan(*map(d64, (x, dt, mild, B, C)), cu.cpu(), d64(D), d64(z), softplus=False, seg=32)
    within(y, (want.y, want.ey), "y")
    within(state, (want.end, want.eend), "state")
    dy = randn(g, n, d, io=IO[io])
    got = ssd.ssd_selective_scan_bwd(x, dt, A, B, C, cu, dy, kept, D, z, softplus=False)
    ssd.ssd_get_device_status()
    grads = want.bwd(d64(dy))
    for k in ("dx", "ddt", "dA", "dB", "dC", "dz"):
        within(got[k], grads[k], k)


# ------------------------------------------------------------------------ norms

MANY = 2400  # rows (or groups) from which on a thread takes more of a row


def some_rows(rows, g):
    return torch.cat([torch.tensor([0, 1, rows - 1]), torch.randint(rows, (30,), generator=g)])


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("width,pad", [(256, 8), (512, 0), (520, 0), (1024, 8), (2048, 0), (4096, 8), (8192, 0), (100, 0), (127, 1), (333, 0),
                                       (1333, 1), (2047, 0), (2049, 1), (8191, 0), (1002, 2), (1332, 2), (4004, 2), (8190, 2)])
def test_norm_before_of_many_rows(io, res, width, pad):
    g, io, res = gen(width), IO[io], IO[res]
    x, r0 = strided(randn(g, MANY, width, io=io), pad), strided(randn(g, MANY, width, io=res, scale=3.0), pad)
    w, s = 1 + randn(g, width, scale=0.1), torch.rand(width, generator=g).cuda()
    at = some_rows(MANY, g)
    for scale in (s, None):
        out, r = ssd.ssd_residual_rmsnorm(x, w, r0, scale)
        pick = lambda t: d64(t[at.cuda()])  # noqa: E731
        want, wr, mo, mr = ref.norm_before(pick(x), d64(w), pick(r0), d64(scale))
        close(out[at.cuda()], want, mo, NORM_ROUNDINGS, "out")
        close(r[at.cuda()], wr, mr, 4, "r")
    few = ssd.ssd_residual_rmsnorm(x[:7], w, r0[:7], None)[0]  # another split of the same rows
    assert ((few.double() - out[:7].double()).abs() <= torch.finfo(io).eps * few.double().abs() + 2 * NORM_ROUNDINGS * 2.0 ** -24 * few.double().abs()).all()
    ssd.ssd_get_device_status()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,G,per,pad", [(MANY, 1, 256, 8), (310, 8, 512, 0), (310, 8, 1024, 8), (MANY, 1, 2048, 0), (310, 8, 333, 1),
                                            (310, 8, 100, 0), (310, 8, 1002, 2), (MANY, 1, 4004, 2), (MANY, 1, 8191, 1), (1200, 2, 8192, 0),
                                            (2500, 1, 127, 0), (900, 3, 1333, 1)])
@pytest.mark.parametrize("first", [False, True])
def test_norm_after_of_many_groups(io, rows, G, per, pad, first):
    g, io, width = gen(per + G), IO[io], G * per
    y, z, r0 = (strided(randn(g, rows, width, io=io), pad) for _ in range(3))
    w, s = 1 + randn(g, width, scale=0.1), torch.rand(width, generator=g).cuda()
    at = some_rows(rows, g)
    out = ssd.ssd_gated_rmsnorm(y, z, w, r0, s, ngroups=G, norm_before_gate=first)
    ssd.ssd_get_device_status()
    pick = lambda t: d64(t[at.cuda()])  # noqa: E731
    want, mag = ref.norm_after(pick(y), pick(z), d64(w), pick(r0), d64(s), G, first)
    close(out[at.cuda()], want, mag, NORM_ROUNDINGS, "out")


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("width", [514, 1002, 1332, 2050, 4002, 4100, 5002, 5120, 8190, 8191])
def test_norm_before_gradients_of_pairs_and_wide_rows(io, res, width):
    g, io, res, rows = gen(width), IO[io], IO[res], 61
    x, r = strided(randn(g, rows, width, io=io), 2), strided(randn(g, rows, width, io=res), 2)
    w, s = 1 + randn(g, width, scale=0.1), torch.rand(width, generator=g).cuda()
    dout, dres = randn(g, rows, width, io=io), randn(g, rows, width, io=res)
    for scale in (s, None):
        want = ref.norm_before_bwd(d64(r), d64(w), d64(dout), d64(dres), d64(x), d64(scale))
        got = ssd.ssd_residual_rmsnorm_bwd(r, w, dout, dres, x, scale)
        for k, (v, m) in want.items():
            close(got[k], v, m, NORM_ROUNDINGS + (rows if k in ("dweight", "dscale") else 0), k)
    ssd.ssd_get_device_status()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("G,per", [(1, 514), (2, 1002), (1, 1332), (3, 2050), (1, 4100), (1, 5002), (2, 5120), (1, 8190), (1, 8191)])
@pytest.mark.parametrize("first", [False, True])
def test_norm_after_gradients_of_pairs_and_wide_groups(io, G, per, first):
    g, io, rows, width = gen(per + G), IO[io], 61, G * per
    y, z = (strided(randn(g, rows, width, io=io), 2) for _ in range(2))
    w, s, dout = 1 + randn(g, width, scale=0.1), torch.rand(width, generator=g).cuda(), randn(g, rows, width, io=io)
    for scale in (s, None):
        want = ref.norm_after_bwd(d64(y), d64(z), d64(w), d64(dout), d64(scale), G, first)
        got = ssd.ssd_gated_rmsnorm_bwd(y, z, w, dout, scale, ngroups=G, norm_before_gate=first)
        for k, (v, m) in want.items():
            close(got[k], v, m, NORM_ROUNDINGS + (rows if k in ("dweight", "dscale") else 0), k)
    ssd.ssd_get_device_status()
