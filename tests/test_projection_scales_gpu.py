"""Scales of the product of 8-bit operands over the range that it takes: two scales whose product is a finite fp32 number,
however large or small each of them is, on every plan of a launch.
"""
import pytest
import torch

import projection_ref as R
from test_projection_gpu import BF, F32, TILES, Rand, inside, ssm, tolerance

pytestmark = pytest.mark.gpu

# workgroups that share k (16, 32 and 64 rows of a), then tiles of every kind
PLANS = [(13, 200, 272, BF), (29, 200, 272, F32), (300, 300, 1168, F32)] + TILES


def powers(r, lo, hi, *shape):
    return torch.exp2(torch.randint(lo, hi, shape, generator=r.g, device="cuda").float()) * (1 + torch.rand(*shape, generator=r.g, device="cuda"))


@pytest.mark.parametrize("b_rows", [128, 1], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,N,K,out", PLANS)
def test_scales_far_apart(M, N, K, out, b_rows):
    """One scale near 2^118, the other near 2^-118, either way round: the sum of a block (2^17 for codes drawn evenly, 2^24 at
    most) times the large one alone is out of fp32's range, the scales' product is an ordinary number."""
    r = Rand(M + N + K)
    blocks = (K + 127) // 128
    a, b = r.codes(M, K), r.codes(N, K)
    for lo in (116, -120):
        sa, sb = powers(r, lo, lo + 4, M, blocks), powers(r, -lo - 4, -lo, -(-N // b_rows), blocks)
        want, size = R.product(a, sa, b, sb, b_rows)
        got = ssm().matmul_fp8(a, sa, b, sb, out_dtype=out)
        inside(got, want, tolerance(a, sa, b, sb, b_rows, out, want, size), "a's scales near 2^%d" % lo)


@pytest.mark.parametrize("b_rows", [128, 1], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,N,K,out", PLANS)
def test_small_products_of_scales(M, N, K, out, b_rows):
    """Products of scales below 2^-126 are fp32 numbers with fewer bits, on every plan the same: each is rounded once, to a
    multiple of 2^-149, and the rest is as ever.  (One block of k, powers of two for a, so that the definition in 64 bits can
    take the rounded products as b's scales.)"""
    r = Rand(M + N + K)
    K = min(K, 128)
    a, b = r.codes(M, K), r.codes(N, K)
    sa, sb = torch.full((M, 1), 2.0 ** -70, device="cuda"), powers(r, -72, -69, -(-N // b_rows), 1)
    rounded = torch.round(sb.double() * 2.0 ** (149 - 70)) * 2.0 ** -149
    want, size = R.product(a, torch.ones_like(sa), b, rounded, b_rows)
    got = ssm().matmul_fp8(a, sa, b, sb, out_dtype=out)
    tol = tolerance(a, torch.ones_like(sa), b, rounded, b_rows, out, want, size)
    # (results below 2^-126 are multiples of 2^-149, or of 2^-133 as bf16)
    inside(got, want, tol + (2.0 ** -134 if out == BF else 2.0 ** -150) * 2, "out")
