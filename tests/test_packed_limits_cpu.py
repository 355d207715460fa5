"""Sizes that the packed operators' C entry points refuse before anything is launched (no GPU needed)."""
import ctypes

import pytest

from test_packed_abi_cpu import FAKE, SHAPE, WORKSPACE, call, conv_params, lib, norm_params, ssd_params  # noqa: F401


@pytest.mark.parametrize("width", [2, 4])
def test_step_needs_a_slot(lib, width):
    """A row without a slot of its own reads the first one's place: there has to be one."""
    assert call(lib, "ssm_conv1d_slot_update", conv_params(nslots=0, width=width)) == SHAPE
    assert lib.ssm_last_error().decode()
