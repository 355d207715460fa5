"""Gradients of the gated norm over groups of few channels, element by element.  There the norm sees little else than the sign
of its input, and dn - nh mean(dn nh) takes away nearly all of dn: what is left is small beside the terms, so it is compared
on their magnitudes."""
import pytest

import packed_ref as R
from test_packed_gpu import BF, Rand, T, f64, ssm, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, "first", "behind"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("n,groups", [(1, 5), (2, 3), (3, 8), (4, 4), (8, 2), (64, 1)])
def test_gradients_of_small_groups(n, groups, center, gate, dtype):
    torch = T()
    r = Rand(120 + n)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows, D = 37, n * groups
    x, dy = r(rows, D, dtype=dt), r(rows, D, dtype=dt)
    z = r(rows, D, dtype=dt) if gate else None
    w, b = 1 + r(D, scale=0.2), r(D, scale=0.3)
    eps = 1e-2
    got = ssm().gated_norm_bwd(x, w, dy, b, z, groups=groups, eps=eps, gate_first=gate == "first", center=center)
    torch.cuda.synchronize()
    X, W, Bb, Z, G = f64(x), f64(w), f64(b), f64(z), f64(dy)
    ref = R.norm_grads(X, W, Bb, Z, groups, eps, gate == "first", center, G)
    s, sl = (R.silu(Z), R.silu_slope(Z)) if gate else (None, None)
    h = (X * s if gate == "first" else X).reshape(rows, groups, n)
    big = h.abs() + (h.abs().mean(-1, keepdim=True) if center else 0)         # what h is the difference of
    if center:
        h = h - h.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    dn = ((G * s if gate == "behind" else G) * W).reshape(rows, groups, n)
    nh = big * rstd
    # dh = rstd (dn - nh mean(dn nh) - mean(dn)); nh carries the roundings of h (its gate's silu, 2^-20, and the mean's) over
    # rstd, and so do the statistics: each of the three terms is off by 2^-17 at most, of the magnitudes
    dh = (rstd * (dn.abs() + nh * (dn.abs() * nh).mean(-1, keepdim=True) + (dn.abs().mean(-1, keepdim=True) if center else 0)))
    # (an error in h moves rstd by rstd^2 times its mean with nh)
    dh = (dh * (1 + (nh * nh).mean(-1, keepdim=True))).reshape(rows, D)
    half = BF if dt.itemsize == 2 else 2.0 ** -24
    flat = nh.reshape(rows, D)
    mag = {"dx": dh * s.abs() if gate == "first" else dh}
    if gate == "first":
        mag["dz"] = dh * X.abs() * (sl.abs() + 1)
    elif gate:
        mag["dz"] = G.abs() * (flat * (1 + (nh * nh).mean(-1, keepdim=True)).expand_as(nh).reshape(rows, D) * W.abs() + Bb.abs()) * (sl.abs() + 1)
    for k, m in mag.items():
        within(got[k], half * ref[k].abs() + 2.0 ** -17 * m + 1e-30, ref[k], k)
