"""The mixer-block operators where earlier forms of them went wrong, without a GPU."""
import pytest

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
