"""Sizes that the packed operators' C entry points refuse before anything is launched (no GPU needed)."""
import ctypes

import pytest

from test_packed_abi_cpu import SHAPE, call, conv_params, lib, ssd_params  # noqa: F401


@pytest.mark.parametrize("width", [2, 4])
def test_step_needs_a_slot(lib, width):
    """A row without a slot of its own reads the first one's place: there has to be one."""
    assert call(lib, "ssm_conv1d_slot_update", conv_params(nslots=0, width=width)) == SHAPE
    assert lib.ssm_last_error().decode()


# A launch has fewer than 2^32 threads along a dimension of its grid.
THREADS = 1 << 32


def test_single_tokens_fit_a_launch(lib):
    """1,024 threads (16 for each row of the state) for a token and head."""
    most = THREADS // 1024
    for heads, tokens in ((64, most // 64), (80, 65536), (1, most), (128, 1 << 22)):
        assert call(lib, "ssm_ssd_slot_update", ssd_params(ntokens=tokens, nheads=heads, ngroups=1)) == SHAPE
        assert "launch" in lib.ssm_last_error().decode()


@pytest.mark.parametrize("name", ["ssm_ssd_packed_fwd", "ssm_ssd_packed_bwd"])
def test_sequences_fit_a_launch(lib, name):
    """Workgroups of 512 threads for 4 heads of a group and a segment; every sequence has one."""
    size = getattr(lib, name + "_workspace_bytes")
    for kw in (dict(nseqs=1 << 20, nheads=80, ngroups=1), dict(nseqs=1 << 20, nheads=32, ngroups=8),
               dict(nseqs=1 << 17, nheads=512, ngroups=64)):
        p = ssd_params(ntokens=4096, segment_chunks=4, **kw)
        assert call(lib, name, p) == SHAPE, kw
        assert "work items" in lib.ssm_last_error().decode()
        assert size(ctypes.byref(p)) == 0


def test_backward_fits_a_launch(lib):
    """The main pass has N * 4 threads for a chunk and group, the last sums one for four columns of dB (dC) of a token."""
    size = lib.ssm_ssd_packed_bwd_workspace_bytes
    assert size(ctypes.byref(ssd_params(ntokens=1 << 22, nseqs=1, nheads=64, ngroups=64, dstate=256))) == 0
    assert call(lib, "ssm_ssd_packed_bwd", ssd_params(ntokens=1 << 22, nseqs=1, nheads=64, ngroups=64,
                                                      dstate=256)) == SHAPE
    assert size(ctypes.byref(ssd_params(ntokens=1 << 18, nseqs=1, nheads=64, ngroups=64, dstate=256))) > 0


def test_convolution_fits_a_launch(lib):
    """Workgroups of 256 threads for a tile of at most 64 tokens and for every sequence.  (The backward's have 64: they fit
    at any size that is taken.)"""
    for kw in (dict(nseqs=1 << 24), dict(ntokens=(1 << 30) - 1, dim=8, nseqs=64)):
        assert call(lib, "ssm_conv1d_packed_fwd", conv_params(**kw)) == SHAPE, kw
        assert "launch" in lib.ssm_last_error().decode()
