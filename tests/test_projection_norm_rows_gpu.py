"""The norm over rows of any finite size, over more rows than a launch has workgroups, and in place: against 64 bits, with the
tolerances of the other tests of the norm (additions in a row; u = 2^-24).
"""
import pytest
import torch

import projection_ref as R
from test_projection_gpu import BF, F32, F8, HALF, Rand, additions, inside, ssm, u

pytestmark = pytest.mark.gpu


def check_forward(x, w, residual, eps, what=""):
    T, D = x.shape
    h, y = R.add_norm(x, residual, w, eps)
    got, kept, _ = ssm().add_norm_fwd(x, w, residual, eps=eps)
    # (below 2^-126 values are multiples of 2^-149, as bf16 of 2^-133)
    least = 2.0 ** -149 if x.dtype == F32 else 2.0 ** -133
    inside(got, y, (HALF[x.dtype] + additions(D) * u) * y.abs() + least, what + " y")
    if residual is not None:
        inside(kept, h, (HALF[residual.dtype] + u) * h.abs(), what + " h")
    q, _, scale = ssm().add_norm_fwd(x, w, residual, eps=eps, y_dtype=F8)
    s = R.magnitudes(y, 1).clamp(min=R.LEAST) / R.TOP
    inside(scale, s, (additions(D) + 2) * u * s, what + " scale")
    v = y / R.spread(scale.double(), 1, y.shape)
    inside(q[:, :D], v, R.half_step(v) + (additions(D) + 4) * u * v.abs() * 2, what + " codes")
    assert int(q.view(torch.uint8)[:, D:].count_nonzero()) == 0


def check_backward(h, w, dy, dh, eps, rows, what=""):
    """`rows` behind each other go into a sum of the weight's gradient."""
    T, D = h.shape
    ds, dw, size, dwsize = R.add_norm_grads(h, w, dy, dh, eps)
    g = ssm().add_norm_bwd(h, w, dy, dh, eps=eps)
    for k in ("dx", "dresidual"):
        least = 2.0 ** -149 if g[k].dtype == F32 else 2.0 ** -133
        inside(g[k], ds, HALF[g[k].dtype] * ds.abs() + 2 * additions(D) * u * size + least, what + " " + k)
    # (a lane adds the rows of its turns, a workgroup its 4 teams, a second kernel 32 runs of workgroups, 16 in each, and those)
    inside(g["dweight"], dw, (additions(D) + rows + 4 + 512 / 32 + 32) * u * dwsize, what + " dweight")


# Teams of one, four and sixteen waves; several turns of the workgroups (16384, 4096 and 1024 rows a turn), the last one cut
@pytest.mark.parametrize("T,D,dtype,res", [(16391, 200, BF, F32), (33001, 72, F32, None), (4099, 2560, BF, F32), (9001, 1100, BF, BF),
                                           (1030, 8200, BF, F32), (2051, 16380, BF, BF), (16390, 777, F32, BF)])
def test_more_rows_than_workgroups(T, D, dtype, res):
    r = Rand(T + D)
    x, w = r(T, D, dtype=dtype, wide=4), 1 + r(D, scale=0.2)
    check_forward(x, w, None if res is None else r(T, D, scale=2.0, dtype=res), 1e-5)


# (512 workgroups of four teams of one wave or one of four, 256 of one team of sixteen)
@pytest.mark.parametrize("T,D,dtype,htype,rows", [(300, 8200, BF, F32, 2), (777, 16381, F32, BF, 4), (4101, 333, BF, BF, 3),
                                                  (1500, 4000, BF, F32, 3)])
def test_gradients_of_more_rows_than_workgroups(T, D, dtype, htype, rows):
    r = Rand(T + D)
    check_backward(r(T, D, scale=2.0, dtype=htype), 1 + r(D, scale=0.2), r(T, D, dtype=dtype, wide=2), r(T, D, dtype=htype), 1e-5, rows)


# Channels of one, four and sixteen waves, cut chunks and whole ones.
SIZES = [1, 64, 520, 1001, 2560, 8192, 16379]


@pytest.mark.parametrize("power", [126, 90, 63, 55, 40, -40])
@pytest.mark.parametrize("D", SIZES)
def test_rows_of_any_size(D, power):
    """Rows whose squares leave fp32's range, between rows of ordinary ones."""
    r = Rand(D + power)
    T = 9
    size = torch.ones(T, 1, device="cuda", dtype=torch.float64)
    size[1::3] = 2.0 ** power
    w = 1 + r(D, scale=0.2)
    for dtype in (BF, F32):
        x = (r(T, D).clamp(-1.9, 1.9).double() * size).to(dtype)
        check_forward(x, w, None, 1e-5)
        check_forward(x, w, (x.double() * 0.5).float(), 1e-5)
        for htype in (BF, F32):
            dy = r(T, D, dtype=dtype)
            check_backward(x.to(htype), w, dy, None, 1e-5, 3)
            check_backward(x.to(htype), w, dy, r(T, D, dtype=htype), 1e-5, 3)


@pytest.mark.parametrize("power", [-60, -75, -100])
@pytest.mark.parametrize("D", SIZES)
def test_small_rows_without_eps(D, power):
    """eps = 0 and rows whose squares are below fp32's range."""
    r = Rand(D - power)
    T = 9
    size = torch.ones(T, 1, device="cuda", dtype=torch.float64)
    size[1::3] = 2.0 ** power
    w = 1 + r(D, scale=0.2)
    for dtype in (BF, F32):
        x = (r(T, D).double() * size).to(dtype)
        check_forward(x, w, None, 0.0)
        # (of one channel the gradient is the difference of two equal numbers, 1 / h in size)
        check_backward(x, w, (r(T, D).double() * size).to(dtype), None, 0.0, 3)


def test_largest_values():
    """The largest finite value of either type, in one channel and in all of them."""
    w = torch.ones(2560, device="cuda")
    for dtype in (BF, F32):
        top = torch.finfo(dtype).max
        x = torch.zeros(3, 2560, device="cuda", dtype=dtype)
        x[0, 7], x[1], x[2] = -top, top, 1.0
        y, _, _ = ssm().add_norm_fwd(x, w)
        want = R.add_norm(x, None, w, 1e-5)[1]
        inside(y, want, (HALF[dtype] + additions(2560) * u) * want.abs())
        big = torch.full((3, 2560), 3.0e38, device="cuda")
        y, h, _ = ssm().add_norm_fwd(big, w, big)                # the sum itself is out of range: infinite, and no norm
        assert h.isinf().all() and y.isnan().all()


def test_in_place_of_x():
    """residual_out may be x where the types agree, with and without a residual, and the gradient may take h's place."""
    r = Rand(8)
    for D in (200, 1001, 2560, 9000):
        x, res, w = r(37, D), r(37, D), 1 + r(D, scale=0.1)
        y, h, _ = ssm().add_norm_fwd(x, w, res)
        x2 = x.clone()
        y2, h2, _ = ssm().add_norm_fwd(x2, w, res, residual_out=x2)
        assert h2 is x2 and torch.equal(y2, y) and torch.equal(h2, h)
        x2 = x.clone()
        y3, h3, _ = ssm().add_norm_fwd(x2, w, residual_out=x2)
        assert h3 is x2 and torch.equal(h3, x) and torch.equal(y3, ssm().add_norm_fwd(x, w)[0])
        dy = r(37, D)
        g = ssm().add_norm_bwd(h, w, dy, res)
        h2 = h.clone()
        g2 = ssm().add_norm_bwd(h2, w, dy, res, dresidual=h2)
        assert g2["dresidual"] is h2 and torch.equal(h2, g["dresidual"]) and torch.equal(g2["dweight"], g["dweight"])
