"""The mixer-block operators where earlier forms of them went wrong, without a GPU."""
import types

import pytest
import torch

import mixer_ref as ref
import selective_state_space_22_b200 as ssd
from mixer_bounds import Scan
from selective_state_space_22_b200 import build as ssd_build

FAKE = 1 << 20  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load_library()


def test_slots_of_a_conv_without_states_are_checked_too(lib):
    update = lambda slots, K: lib.ssd_conv1d_update(None, slots, FAKE, 12, FAKE, None, FAKE, None, None, 0, 5, 0, 12, 0, K, 1, None)  # noqa: E731
    assert update(FAKE + 2, 1) == ssd.SSD_ERR_INVALID_ARG and "slots" in ssd.ssd_last_error()
    assert update(FAKE, 2) == ssd.SSD_ERR_INVALID_ARG and "conv_state" in ssd.ssd_last_error()  # two taps need one


def test_one_array_for_two_different_gradients_is_refused(lib):
    def bwd(io, rio, scale, dx, dres):
        s = FAKE if scale else None
        return lib.ssd_residual_rmsnorm_bwd(FAKE, 8, FAKE, FAKE, None, s, 8, s, dx, dres, FAKE, s, io, rio, 4, 8, 1e-5, None, 0, None)

    for io, rio, scale in ((0, 0, True), (1, 0, False), (1, 1, True)):
        assert bwd(io, rio, scale, FAKE, FAKE) == ssd.SSD_ERR_INVALID_ARG and "one array" in ssd.ssd_last_error()
        assert bwd(io, rio, scale, FAKE, FAKE + 4096) == ssd.SSD_ERR_WORKSPACE  # the next check
    assert bwd(0, 0, False, FAKE, FAKE) == ssd.SSD_ERR_WORKSPACE


def test_a_stream_of_another_device_is_refused():
    """It would be replaced by the tensors' device's own stream, which nobody waits for."""
    at = lambda k: types.SimpleNamespace(device=torch.device("cuda", k))  # noqa: E731
    x, w = at(0), at(0)
    for call in (lambda: ssd.ssd_conv1d_varlen(x, w, None, w, stream=at(1)), lambda: ssd.ssd_conv1d_update(w, x, w, stream=at(1)),
                 lambda: ssd.ssd_conv1d_bwd(x, w, None, w, w, stream=at(1)), lambda: ssd.ssd_selective_scan_varlen(x, w, w, w, w, w, stream=at(1)),
                 lambda: ssd.ssd_selective_state_update(w, x, w, w, w, w, stream=at(1)),
                 lambda: ssd.ssd_selective_scan_bwd(x, w, w, w, w, w, w, w, stream=at(1)), lambda: ssd.ssd_residual_rmsnorm(x, w, stream=at(1)),
                 lambda: ssd.ssd_residual_rmsnorm_bwd(x, w, w, stream=at(1)), lambda: ssd.ssd_gated_rmsnorm(x, w, w, stream=at(1)),
                 lambda: ssd.ssd_gated_rmsnorm_bwd(x, w, w, w, stream=at(1))):
        with pytest.raises(ValueError, match="stream is on cuda:1, the tensors are on cuda:0"):
            call()


def test_the_binding_is_built_again_for_another_torch(lib, monkeypatch):
    assert not ssd_build._bind_stale()
    mine = ssd_build._bind_for()
    assert torch.__version__.split("+")[0] in mine
    monkeypatch.setattr(ssd_build, "_bind_for", lambda: mine.replace("torch ", "torch 9"))
    assert ssd_build._bind_stale()
    monkeypatch.undo()
    monkeypatch.setattr(ssd_build, "BIND_FOR", ssd_build.BIND_FOR + ".missing")
    assert ssd_build._bind_stale()


@pytest.mark.parametrize("softplus", [True, False])
def test_the_bounded_formulas_are_the_formulas(softplus):
    """mixer_bounds.Scan has mixer_ref's values, and its bounds hold a float32 evaluation
    without being longer than a few hundred roundings of what is summed."""
    g, n, d, G, N = torch.Generator().manual_seed(3), 60, 12, 2, 5
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, dt, A, B, C, dy = r(n, d), r(n, d), -torch.rand(d, N, generator=g) * 15 - 1, r(n, G, N), r(n, G, N), r(n, d)
    cu, opt = torch.tensor([0, 25, 25, 26, 60]), (r(d), r(n, d), r(d) * 0.5 - 2.5) if softplus else (None, None, None)
    dt = dt if softplus else dt.abs() * 0.1
    d64 = ref.d64
    ins, opt64 = [d64(t) for t in (x, dt, A, B, C)], [d64(t) for t in opt]
    scan = Scan(*ins, cu, *opt64, softplus=softplus)
    y, mag, end, mend, _ = ref.sel(*ins, cu, *opt64, softplus=softplus)
    assert torch.allclose(scan.y, y, rtol=1e-12) and torch.allclose(scan.end, end, rtol=1e-12)
    assert (scan.ey <= 500 * mag).all() and (scan.eend <= 500 * mend).all()
    want = ref.sel_bwd(*ins, cu, d64(dy), *opt64, softplus=softplus)
    for k, (v, e) in scan.bwd(d64(dy)).items():
        assert torch.allclose(v, want[k][0], rtol=1e-11, atol=1e-13), k
        assert (e <= 2000 * want[k][1] + 1e-30).all(), k
    h, delta = torch.zeros(d, N), torch.nn.functional.softplus(dt + opt[2]) if softplus else dt  # in float32
    for t in range(25):
        h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * B[t].repeat_interleave(d // G, 0)
    assert ((h.double() - scan.end[0]).abs() <= ref.U32 * scan.eend[0]).all()
