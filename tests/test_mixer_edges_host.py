"""The mixer-block operators where earlier forms of them went wrong, without a GPU."""
import types

import pytest
import torch

import selective_state_space_22_b200 as ssd
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
