"""What the 8-bit matrix instructions drop of a bf16 result: at most 5e-5 of the results' 2-norm, as the header says, on every
plan of a launch.

The results' own rounding (1.7e-3) covers that, so the results are compared with the correctly rounded ones.  With e = (what
was dropped), w = the exact result and s = the distance of the bf16 values around it, w + e and w round to values that are
apart by n s or (n + 1) s where |e| = (n + f) s, the second in a share f of the cases (the border lies anywhere between the
values): the square of that is s^2 (n^2 + (2 n + 1) f) on average, at most e^2 + |e| s.  s <= 2^-7 |w|, so over all results
(sums by Cauchy and Schwarz) the difference is at most sqrt(r^2 + 2^-7 r) of the 2-norm for r = |e| / |w| = 5e-5: 6.3e-4.  The
fp32 sums around the instructions add 2^-24 for each of up to 2 blocks + 12 additions to r, below 1e-5.
"""
import pytest
import torch

import projection_ref as R
from test_projection_gpu import BF, F32, TILES, Rand, ssm

pytestmark = pytest.mark.gpu

DROPPED = 5e-5
# workgroups that share k (16, 32 and 64 rows of a, and 96 of b), then tiles of every kind
PLANS = [(16, 10576, 2560), (32, 3352, 768), (61, 5120, 2560), (510, 2557, 2320)] + [(m, n, max(k, 400)) for m, n, k, out in TILES if out == BF]


def operands(r, M, N, K, b_rows, kind):
    blocks = (K + 127) // 128
    if kind == "codes":     # any codes, evenly
        return r.codes(M, K), r.scales(M, blocks), r.codes(N, K), r.scales(-(-N // b_rows), blocks)
    # activations with larger channels among them, and a weight
    x, w = r(M, K) * torch.exp(r(1, K)), r(N, K, scale=K ** -0.5)
    xq, wq = ssm().quantize_fp8(x), (ssm().quantize_fp8_blocks if b_rows == 128 else ssm().quantize_fp8)(w)
    return xq["q"], xq["scale"], wq["q"], wq["scale"]


@pytest.mark.parametrize("kind", ["codes", "values"])
@pytest.mark.parametrize("b_rows", [128, 1], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,N,K", PLANS)
def test_dropped(M, N, K, b_rows, kind):
    a, sa, b, sb = operands(Rand(M + N + K), M, N, K, b_rows, kind)
    want, _ = R.product(a, sa, b, sb, b_rows)
    got = ssm().matmul_fp8(a, sa, b, sb)
    r = DROPPED + (2 * ((K + 127) // 128) + 12) * 2.0 ** -24
    share = float((got.double() - want.to(BF).double()).norm() / want.norm())
    print("of the correctly rounded results' 2-norm: %.2e" % share)
    assert share <= (r * r + 2.0 ** -7 * r) ** 0.5


@pytest.mark.parametrize("M,N", [(5, 40), (100, 300), (2100, 2600)])
def test_large_products_that_cancel(M, N):
    """Products that cancel in a block: an fp32 result keeps what is left, exactly; a bf16 one is off by 2^-12 of them for each
    of the groups that an instruction adds up, and no more."""
    r = Rand(M)
    K = 256
    a = torch.randint(-3, 4, (M, K), generator=r.g, device="cuda").float()
    b = torch.randint(-3, 4, (N, K), generator=r.g, device="cuda").float()
    a[:, 3], a[:, 77], b[:, 3], b[:, 77] = 448.0, 448.0, 448.0, -448.0
    one = torch.ones(M, 2, device="cuda"), torch.ones(-(-N // 128), 2, device="cuda")
    want = a.double() @ b.double().T
    a, b = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    assert torch.equal(ssm().matmul_fp8(a, one[0], b, one[1], out_dtype=F32).double(), want)
    off = (ssm().matmul_fp8(a, one[0], b, one[1]).double() - want).abs()
    assert bool((off <= 2.0 ** -8 * want.abs() + 16 * 2.0 ** -12 * 448.0 ** 2).all())
