"""Refusals of the packed operators' C entry points and of their Python forms: each is checked before anything is
launched, so these calls never reach the HIP runtime and run without a GPU."""
import ctypes

import pytest
import torch

import selective_state_space_57_amd as ssm
from selective_state_space_57_amd import _abi

FAKE = 0x10000   # a non-NULL, 256-byte aligned address, never dereferenced
NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def lib():
    return _abi.lib()


def conv_params(**kw):
    base = dict(ntokens=100, nseqs=3, dim=40, nslots=4, width=4, activation=1, io_dtype=_abi.SSM_BF16)
    return _abi.ConvPackedParams(**{**base, **kw})


def ssd_params(**kw):
    base = dict(ntokens=100, nseqs=3, nheads=6, headdim=64, ngroups=2, dstate=128, nslots=4, io_dtype=_abi.SSM_BF16,
                disc=0, dt_softplus=1)
    return _abi.SsdPackedParams(**{**base, **kw})


def norm_params(**kw):
    base = dict(ntokens=100, dim=40, ngroups=2, eps=1e-5, io_dtype=_abi.SSM_BF16, gate_first=1)
    return _abi.GatedNormParams(**{**base, **kw})


# an entry point: its pointers in order, the ones that are required, and whether a workspace follows
ENTRIES = {
    "ssm_conv1d_packed_fwd": (conv_params, "x weight bias cu state idx has state_out u", "x weight cu u", False),
    "ssm_conv1d_slot_update": (conv_params, "x weight bias state idx u", "x weight state u", False),
    "ssm_conv1d_packed_bwd": (conv_params, "x weight bias cu state idx has du dstate_out dx dweight dbias dstate",
                              "x weight cu du dx dweight", True),
    "ssm_ssd_packed_fwd": (ssd_params, "x dt dt_bias A B C Dskip cu state idx has state_out y", "x dt A B C cu y", True),
    "ssm_ssd_packed_bwd": (ssd_params, "x dt dt_bias A B C Dskip cu state idx has dy dstate_out dx ddt dA dB dC dDskip "
                           "ddt_bias dstate", "x dt A B C cu dy dx ddt dA dB dC", True),
    "ssm_ssd_slot_update": (ssd_params, "state x dt dt_bias A B C Dskip idx y", "state x dt A B C y", False),
    "ssm_gated_norm_fwd": (norm_params, "x z weight bias y", "x weight y", False),
    "ssm_gated_norm_bwd": (norm_params, "x z weight bias dy dx dz dweight dbias", "x weight dy dx dweight", True),
}


def call(lib, name, params, ws=0, ws_bytes=0, **ptrs):
    make, names, required, space = ENTRIES[name]
    args = [ptrs.get(n, FAKE if n in required.split() else 0) for n in names.split()]
    args += [ws, ws_bytes] if space else []
    return getattr(lib, name)(None if params is None else ctypes.byref(params), *args, 0)


@pytest.mark.parametrize("name", ENTRIES)
def test_null_params_and_pointers(lib, name):
    make, _, required, _ = ENTRIES[name]
    assert call(lib, name, None) == NULL
    for n in required.split():
        assert call(lib, name, make(), **{n: 0}) == NULL, n
    assert lib.ssm_last_error().decode()


BAD = {
    conv_params: [(dict(ntokens=0), SHAPE), (dict(ntokens=1 << 30), SHAPE), (dict(dim=0), SHAPE),
                  (dict(dim=1 << 24), SHAPE), (dict(nslots=-1), SHAPE), (dict(width=0), SHAPE), (dict(width=5), SHAPE),
                  (dict(x_stride=39), SHAPE), (dict(u_stride=-1), SHAPE), (dict(activation=2), UNSUPPORTED),
                  (dict(io_dtype=9), DTYPE), (dict(reserved=1), UNSUPPORTED)],
    ssd_params: [(dict(ntokens=0), SHAPE), (dict(ntokens=1 << 30), SHAPE), (dict(nheads=0), SHAPE),
                 (dict(ngroups=0), SHAPE), (dict(ngroups=4), SHAPE), (dict(headdim=32), UNSUPPORTED),
                 (dict(dstate=96), UNSUPPORTED), (dict(nslots=-1), SHAPE), (dict(io_dtype=_abi.SSM_F32), DTYPE),
                 (dict(disc=7), UNSUPPORTED), (dict(dt_softplus=2), UNSUPPORTED), (dict(segment_chunks=-1), UNSUPPORTED),
                 (dict(x_stride=6 * 64 - 1), SHAPE), (dict(b_stride=1 << 24), SHAPE), (dict(dt_stride=5), SHAPE),
                 (dict(reserved=1), UNSUPPORTED)],
    norm_params: [(dict(ntokens=0), SHAPE), (dict(dim=0), SHAPE), (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE),
                  (dict(dim=16385, ngroups=1), UNSUPPORTED), (dict(io_dtype=5), DTYPE), (dict(gate_first=2), UNSUPPORTED),
                  (dict(center=-1), UNSUPPORTED), (dict(x_stride=39), SHAPE), (dict(dz_stride=-40), SHAPE),
                  (dict(reserved=1), UNSUPPORTED)],
}


@pytest.mark.parametrize("name", ENTRIES)
def test_parameters(lib, name):
    make = ENTRIES[name][0]
    for kw, code in BAD[make]:
        assert call(lib, name, make(**kw)) == code, kw
    if make is not norm_params and "slot" not in name:
        assert call(lib, name, make(nseqs=0)) == SHAPE
        assert call(lib, name, make(nseqs=1 << 30)) == SHAPE
    if make is norm_params:
        for eps in (-1.0, float("nan")):
            assert call(lib, name, make(eps=eps)) in (SHAPE, UNSUPPORTED), eps
    size = getattr(lib, name + "_workspace_bytes", None)
    if size is not None:
        assert size(None) == 0
        for kw, _ in BAD[make]:
            assert size(ctypes.byref(make(**kw))) == 0, kw


def test_step_refuses_more_rows_than_a_grid_has(lib):
    assert call(lib, "ssm_conv1d_slot_update", conv_params(ntokens=65536)) == SHAPE
    assert call(lib, "ssm_ssd_slot_update", ssd_params(nslots=0)) == SHAPE


@pytest.mark.parametrize("name,ptr,off", [
    ("ssm_conv1d_packed_fwd", "x", 1), ("ssm_conv1d_packed_fwd", "weight", 2), ("ssm_conv1d_packed_fwd", "cu", 2),
    ("ssm_conv1d_packed_fwd", "state_out", 2), ("ssm_conv1d_slot_update", "u", 1), ("ssm_conv1d_packed_bwd", "dx", 1),
    ("ssm_conv1d_packed_bwd", "dstate_out", 2),
    ("ssm_ssd_packed_fwd", "x", 8), ("ssm_ssd_packed_fwd", "B", 2), ("ssm_ssd_packed_fwd", "y", 4),
    ("ssm_ssd_packed_fwd", "state", 4), ("ssm_ssd_packed_fwd", "dt", 1), ("ssm_ssd_packed_fwd", "cu", 2),
    ("ssm_ssd_packed_bwd", "dy", 8), ("ssm_ssd_packed_bwd", "dB", 4), ("ssm_ssd_packed_bwd", "dstate", 8),
    ("ssm_ssd_packed_bwd", "dA", 2), ("ssm_ssd_slot_update", "state", 8), ("ssm_ssd_slot_update", "C", 4),
    ("ssm_gated_norm_fwd", "x", 1), ("ssm_gated_norm_fwd", "weight", 2), ("ssm_gated_norm_bwd", "dbias", 2)])
def test_alignment(lib, name, ptr, off):
    assert call(lib, name, ENTRIES[name][0](), **{ptr: FAKE + off}) == ALIGN
    assert lib.ssm_last_error().decode()


@pytest.mark.parametrize("name,field", [("ssm_ssd_packed_fwd", "x_stride"), ("ssm_ssd_packed_fwd", "y_stride"),
                                        ("ssm_ssd_packed_bwd", "dx_stride")])
def test_row_strides_off_16_bytes(lib, name, field):
    assert call(lib, name, ssd_params(**{field: 6 * 64 + 4})) == ALIGN


@pytest.mark.parametrize("name,kw", [
    ("ssm_conv1d_packed_bwd", {}), ("ssm_conv1d_packed_bwd", dict(dim=7, io_dtype=_abi.SSM_F32)),
    ("ssm_ssd_packed_fwd", dict(ntokens=20000)), ("ssm_ssd_packed_fwd", dict(ntokens=20000, segment_chunks=1)),
    ("ssm_ssd_packed_bwd", {}), ("ssm_ssd_packed_bwd", dict(ntokens=20000)), ("ssm_gated_norm_bwd", {}),
    ("ssm_gated_norm_bwd", dict(ntokens=70000, dim=5120))])
def test_workspace(lib, name, kw):
    p = ENTRIES[name][0](**kw)
    need = getattr(lib, name + "_workspace_bytes")(ctypes.byref(p))
    assert need > 0
    assert call(lib, name, p) == WORKSPACE
    assert call(lib, name, p, ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert call(lib, name, p, ws=0, ws_bytes=need) == WORKSPACE
    assert call(lib, name, p, ws=FAKE + 2, ws_bytes=need) == WORKSPACE


def test_gate_gradient_goes_with_the_gate(lib):
    assert call(lib, "ssm_gated_norm_bwd", norm_params(), z=FAKE) == NULL
    assert call(lib, "ssm_gated_norm_bwd", norm_params(), dz=FAKE) == NULL


def test_one_chunk_runs_need_no_workspace(lib):
    size = lib.ssm_ssd_packed_fwd_workspace_bytes
    assert size(ctypes.byref(ssd_params(ntokens=64, nseqs=1))) == 0
    # a forced length of 1: a state of H x 64 x N and a decay for each of at most ntokens / 64 + nseqs runs
    assert size(ctypes.byref(ssd_params(ntokens=6400, nseqs=1, segment_chunks=1))) >= 99 * 6 * 64 * 128 * 4
    assert size(ctypes.byref(ssd_params(ntokens=6400, nseqs=1, segment_chunks=100))) == 0


def test_workspace_does_not_grow_with_short_sequences(lib):
    """Only sequences of several segments need their states kept between passes: at most two places for every whole
    segment of the tokens."""
    size = lib.ssm_ssd_packed_fwd_workspace_bytes
    state = 6 * 64 * 128 * 4
    for nseqs in (1, 100, 16384):
        p = ssd_params(ntokens=16384, nseqs=nseqs, segment_chunks=4)
        assert size(ctypes.byref(p)) <= 2 * (16384 // 256) * (state + 6 * 4) + 512, nseqs


def test_python_forms_want_the_gpu():
    """Tensors in host memory are refused before the library is called."""
    x, w, cu = torch.zeros(4, 8), torch.zeros(8, 4), torch.tensor([0, 4], dtype=torch.int32)
    h, g = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    d, A = torch.zeros(4, 2, dtype=torch.bfloat16), torch.zeros(2)
    for f in (lambda: ssm.conv1d_packed_fwd(x, w, cu), lambda: ssm.conv1d_packed_bwd(x, w, x, cu),
              lambda: ssm.conv1d_slot_update(torch.zeros(4, 8, 3), x, w),
              lambda: ssm.ssd_packed_fwd(h, d, A, g, g, cu), lambda: ssm.ssd_packed_bwd(h, d, A, g, g, h, cu),
              lambda: ssm.ssd_slot_update(torch.zeros(4, 2, 64, 64), h, d, A, g, g),
              lambda: ssm.gated_norm_fwd(x, torch.ones(8)), lambda: ssm.gated_norm_bwd(x, torch.ones(8), x)):
        with pytest.raises(ValueError, match="GPU"):
            f()
