"""What the C entry points at a block's ends say of their parameters, where no GPU is needed to see it: the parameters of a
forward call serve its backward too."""
import ctypes

import pytest

from selective_state_space_57_amd import _abi
from test_projection_abi_cpu import DTYPE, FAKE, WORKSPACE, call, norm_params


@pytest.fixture(scope="module")
def lib():
    return _abi.lib()


@pytest.mark.parametrize("io", [_abi.SSM_F32, _abi.SSM_BF16])
def test_types_of_y_in_the_backward(lib, io):
    """The types of y that the forward takes are taken, and change nothing; another one is refused as in the forward."""
    size = lib.ssm_add_norm_bwd_workspace_bytes
    needs = set()
    for y in (io, _abi.SSM_E4M3):
        p = norm_params(io_dtype=io, y_dtype=y)
        needs.add(size(ctypes.byref(p)))
        assert call(lib, "ssm_add_norm_bwd", p) == WORKSPACE     # (all of its parameters have been accepted)
    assert len(needs) == 1 and 0 not in needs
    p = norm_params(io_dtype=io, y_dtype=_abi.SSM_BF16 if io == _abi.SSM_F32 else _abi.SSM_F32)
    assert size(ctypes.byref(p)) == 0
    for name, kw in (("ssm_add_norm_bwd", dict(ws=FAKE, ws_bytes=1 << 30)), ("ssm_add_norm_fwd", {})):
        assert call(lib, name, p, **kw) == DTYPE


def test_the_header_says_so():
    import os
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ssm_scan.h")).read()
    about = text[text.index("Backward of ssm_add_norm_fwd"):text.index("ssm_status ssm_add_norm_bwd(")]
    assert "ignored" not in about and "y_dtype" in about and "refused" in about
