"""Refusals of the C entry points at a block's ends and of their Python forms: each is checked before anything is launched,
so these calls never reach the HIP runtime and run without a GPU."""
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


def norm_params(**kw):
    base = dict(ntokens=100, dim=200, eps=1e-5, io_dtype=_abi.SSM_BF16, res_dtype=_abi.SSM_F32, y_dtype=_abi.SSM_BF16)
    return _abi.AddNormParams(**{**base, **kw})


def norm8_params(**kw):
    return norm_params(**{"y_dtype": _abi.SSM_E4M3, **kw})


def quant_params(**kw):
    return _abi.QuantizeFp8Params(**{**dict(rows=100, cols=200, io_dtype=_abi.SSM_BF16), **kw})


def matmul_params(**kw):
    return _abi.MatmulFp8Params(**{**dict(m=100, n=200, k=256, b_rows=128, out_dtype=_abi.SSM_BF16), **kw})


# an entry point: its pointers in order, the ones that are required, and whether a workspace follows
ENTRIES = {
    "ssm_add_norm_fwd": (norm_params, "x residual weight residual_out y y_scale", "x weight y", False),
    "ssm_add_norm_bwd": (norm_params, "h weight dy dh dx dresidual dweight", "h weight dy dresidual dweight", True),
    "ssm_quantize_fp8": (quant_params, "x q scale qt scale_t", "x q scale", False),
    "ssm_matmul_fp8": (matmul_params, "a a_scale b b_scale out", "a a_scale b b_scale out", False),
}


def call(lib, name, params, ws=0, ws_bytes=0, **ptrs):
    _, names, required, space = ENTRIES[name]
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
    "ssm_add_norm_fwd": [(dict(ntokens=0), SHAPE), (dict(ntokens=1 << 31), SHAPE), (dict(dim=0), SHAPE), (dict(dim=16385), UNSUPPORTED),
                         (dict(io_dtype=2), DTYPE), (dict(res_dtype=2), DTYPE), (dict(y_dtype=0), DTYPE), (dict(y_dtype=3), DTYPE),
                         (dict(eps=-1.0), UNSUPPORTED), (dict(eps=float("nan")), UNSUPPORTED), (dict(x_stride=199), SHAPE),
                         (dict(residual_stride=-1), SHAPE), (dict(h_stride=1), SHAPE), (dict(y_stride=199), SHAPE),
                         (dict(y_dtype=2, y_stride=200), SHAPE), (dict(scale_stride=1), SHAPE), (dict(dy_stride=3), SHAPE),
                         (dict(x_stride=1 << 41), SHAPE), (dict(reserved=1), UNSUPPORTED)],
    "ssm_quantize_fp8": [(dict(rows=0), SHAPE), (dict(cols=0), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(cols=1 << 30), SHAPE),
                         (dict(io_dtype=2), DTYPE), (dict(square=2), UNSUPPORTED), (dict(x_stride=199), SHAPE), (dict(q_stride=192), SHAPE),
                         (dict(scale_stride=1), SHAPE), (dict(qt_stride=96), SHAPE), (dict(rows=(1 << 30) - 1, cols=1 << 20), SHAPE),
                         (dict(reserved=(ctypes.c_int32 * 2)(0, 1)), UNSUPPORTED)],
    "ssm_matmul_fp8": [(dict(m=0), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=24), SHAPE), (dict(m=1 << 30), SHAPE),
                       (dict(n=1 << 30), SHAPE), (dict(k=1 << 23), SHAPE), (dict(a_stride=240), SHAPE), (dict(b_stride=1 << 23), SHAPE),
                       (dict(out_stride=199), SHAPE), (dict(a_scale_stride=1), SHAPE), (dict(b_scale_stride=1 << 20), SHAPE),
                       (dict(b_rows=2), UNSUPPORTED), (dict(out_dtype=2), DTYPE), (dict(reserved=(ctypes.c_int32 * 2)(0, 1)), UNSUPPORTED),
                       (dict(m=(1 << 30) - 1, n=1 << 20), SHAPE), (dict(n=(1 << 30) - 1, m=1), SHAPE)],
}
BAD["ssm_add_norm_bwd"] = [(kw, code) for kw, code in BAD["ssm_add_norm_fwd"] if kw.get("y_dtype") != 0]


@pytest.mark.parametrize("name,kw,code", [(n, kw, code) for n, cases in BAD.items() for kw, code in cases])
def test_params(lib, name, kw, code):
    make = ENTRIES[name][0]
    assert call(lib, name, make(**kw)) == code
    assert lib.ssm_last_error().decode()
    size = getattr(lib, name + "_workspace_bytes", None)
    if size is not None:
        assert size(None) == 0 and size(ctypes.byref(make(**kw))) == 0


@pytest.mark.parametrize("name,ptr,off", [
    ("ssm_add_norm_fwd", "x", 1), ("ssm_add_norm_fwd", "residual", 2), ("ssm_add_norm_fwd", "weight", 2), ("ssm_add_norm_fwd", "y", 1),
    ("ssm_add_norm_fwd", "residual_out", 2), ("ssm_add_norm_bwd", "h", 2), ("ssm_add_norm_bwd", "dy", 1), ("ssm_add_norm_bwd", "dx", 1),
    ("ssm_add_norm_bwd", "dh", 2), ("ssm_add_norm_bwd", "dweight", 2), ("ssm_quantize_fp8", "x", 1), ("ssm_quantize_fp8", "q", 8),
    ("ssm_quantize_fp8", "scale", 2), ("ssm_matmul_fp8", "a", 8), ("ssm_matmul_fp8", "b", 4), ("ssm_matmul_fp8", "a_scale", 2),
    ("ssm_matmul_fp8", "b_scale", 1), ("ssm_matmul_fp8", "out", 1)])
def test_alignment(lib, name, ptr, off):
    assert call(lib, name, ENTRIES[name][0](), **{ptr: FAKE + off}) == ALIGN
    assert lib.ssm_last_error().decode()


def test_alignment_of_8_bit_rows(lib):
    assert call(lib, "ssm_add_norm_fwd", norm8_params(), y=FAKE + 4, y_scale=FAKE) == ALIGN
    assert call(lib, "ssm_add_norm_fwd", norm8_params(y_stride=212), y_scale=FAKE) == ALIGN
    assert call(lib, "ssm_quantize_fp8", quant_params(q_stride=216)) == ALIGN
    assert call(lib, "ssm_quantize_fp8", quant_params(qt_stride=120), qt=FAKE, scale_t=FAKE) == ALIGN
    assert call(lib, "ssm_matmul_fp8", matmul_params(a_stride=264)) == ALIGN
    assert call(lib, "ssm_matmul_fp8", matmul_params(b_stride=260)) == ALIGN


def test_scales_go_with_their_codes(lib):
    assert call(lib, "ssm_add_norm_fwd", norm8_params()) == NULL
    assert call(lib, "ssm_add_norm_fwd", norm_params(), y_scale=FAKE) == NULL
    assert call(lib, "ssm_quantize_fp8", quant_params(), qt=FAKE) == NULL
    assert call(lib, "ssm_quantize_fp8", quant_params(), scale_t=FAKE) == NULL
    assert call(lib, "ssm_quantize_fp8", quant_params(), q=0, scale=0) == NULL


@pytest.mark.parametrize("name,kw", [("ssm_add_norm_bwd", {}), ("ssm_add_norm_bwd", dict(ntokens=70000, dim=5120))])
def test_workspace(lib, name, kw):
    p = ENTRIES[name][0](**kw)
    need = getattr(lib, name + "_workspace_bytes")(ctypes.byref(p))
    assert need > 0
    assert call(lib, name, p) == WORKSPACE
    assert call(lib, name, p, ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert call(lib, name, p, ws=0, ws_bytes=need) == WORKSPACE
    assert call(lib, name, p, ws=FAKE + 2, ws_bytes=need) == WORKSPACE


def test_python_forms_want_the_gpu():
    """Tensors in host memory are refused before the library is called."""
    x, w, q, s = torch.zeros(4, 128), torch.ones(128), torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.ones(4, 1)
    for f in (lambda: ssm.add_norm_fwd(x, w), lambda: ssm.add_norm_bwd(x, w, x), lambda: ssm.quantize_fp8(x),
              lambda: ssm.quantize_fp8_blocks(x), lambda: ssm.matmul_fp8(q, s, q, s)):
        with pytest.raises(ValueError, match="GPU"):
            f()
