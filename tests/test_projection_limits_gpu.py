"""The largest sizes that the operators at a block's ends take: rows, columns and lengths up to their limits, rows as far apart
as they may be.
"""
import pytest
import torch

import projection_ref as R
from test_projection_gpu import BF, F32, F8, HALF, Rand, additions, inside, ssm

pytestmark = pytest.mark.gpu


def room(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip("needs %d GB" % gb)


def whole(r, M, K):
    """Small whole numbers as codes, made in pieces."""
    out = torch.empty(M, K, dtype=F8, device="cuda")
    step = max(1, (1 << 28) // K)
    for i in range(0, M, step):
        n = min(step, M - i)
        out[i:i + n] = torch.randint(-3, 4, (n, K), generator=r.g, device="cuda", dtype=torch.int8).float().to(F8)
    return out


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 33), (29, 50), (70, 130)])
def test_longest_rows(M, N, out):
    """k of 2^23 - 16: whole numbers, whose sums (below 2^24 in every order) are exact."""
    room(16)
    r = Rand(M)
    K = (1 << 23) - 16
    a, b = whole(r, M, K), whole(r, N, K)
    blocks = (K + 127) // 128
    want = torch.zeros(M, N, device="cuda", dtype=torch.float64)
    for c in range(0, K, 1 << 20):
        want += a[:, c:c + (1 << 20)].double() @ b[:, c:c + (1 << 20)].double().T
    got = ssm().matmul_fp8(a, torch.ones(M, blocks, device="cuda"), b, torch.ones(-(-N // 128), blocks, device="cuda"), out_dtype=out)
    assert torch.equal(got, want.to(out))


def test_most_columns():
    """n just below 2^27: workgroups that share k, one row of a."""
    room(16)
    r = Rand(1)
    N, K = (1 << 27) - 80, 16
    a, b = whole(r, 1, K), whole(r, N, K)
    got = ssm().matmul_fp8(a, torch.ones(1, 1, device="cuda"), b, torch.ones(-(-N // 128), 1, device="cuda"))
    for i in range(0, N, 1 << 25):
        assert torch.equal(got[:, i:i + (1 << 25)], (a.float() @ b[i:i + (1 << 25)].float().t()).to(BF))


@pytest.mark.parametrize("M,N,out", [((1 << 30) - 1, 1, BF), ((1 << 27) + 5, 3, BF), ((1 << 27) + 5, 3, F32)])
def test_most_rows(M, N, out):
    """m up to 2^30 - 1: tiles, few columns of them."""
    room(40)
    r = Rand(2)
    K = 16
    a, b = whole(r, M, K), whole(r, N, K)
    got = ssm().matmul_fp8(a, torch.ones(M, 1, device="cuda"), b, torch.ones(1, 1, device="cuda"), out_dtype=out)
    for i in range(0, M, 1 << 26):
        assert torch.equal(got[i:i + (1 << 26)], (a[i:i + (1 << 26)].float() @ b.float().t()).to(out))


@pytest.mark.parametrize("M,N,out,b_rows", [(4099, 2560, BF, 128), (2100, 2600, F32, 1), (2001, 2550, BF, 1)])
def test_rows_far_apart(M, N, out, b_rows):
    """Rows of either operand 2^23 - 16 bytes apart, scales 2^20 - 1, under tiles of 256, 192 and 128 rows."""
    room(80)
    r = Rand(3)
    K, apart, sapart = 272, (1 << 23) - 16, (1 << 20) - 1
    a, b = r.codes(M, K), r.codes(N, K)
    sa, sb = r.scales(M, 3), r.scales(-(-N // b_rows), 3)
    want = ssm().matmul_fp8(a, sa, b, sb, out_dtype=out)

    def spread(t, step):
        base = torch.empty((t.shape[0] - 1) * step + t.shape[1], dtype=t.dtype, device="cuda")
        v = base.as_strided(t.shape, (step, 1))
        v.view(torch.uint8).copy_(t.view(torch.uint8)) if t.dtype == F8 else v.copy_(t)
        return v
    wide = spread(a, apart)
    assert torch.equal(ssm().matmul_fp8(wide, spread(sa, sapart), b, sb, out_dtype=out), want)
    del wide
    assert torch.equal(ssm().matmul_fp8(a, sa, spread(b, apart), spread(sb, sapart), out_dtype=out), want)


def test_norm_of_most_rows():
    """2^31 - 1 rows of one channel."""
    room(40)
    T = (1 << 31) - 1
    x = torch.empty(T, 1, dtype=BF, device="cuda")
    for i in range(0, T, 1 << 28):
        n = min(1 << 28, T - i)
        x[i:i + n, 0] = (torch.arange(i, i + n, device="cuda") % 251 - 100).to(BF)
    w = torch.full((1,), 1.5, device="cuda")
    y, _, _ = ssm().add_norm_fwd(x, w, eps=4.0)
    # (a row's value alone decides its result)
    few = (torch.arange(251, device="cuda") - 100).to(BF)[:, None]
    want = R.add_norm(few, None, w, 4.0)[1]
    got = ssm().add_norm_fwd(few, w, eps=4.0)[0]
    inside(got, want, (HALF[BF] + additions(1) * 2.0 ** -24) * want.abs())
    for i in range(0, T, 1 << 28):
        n = min(1 << 28, T - i)
        assert torch.equal(y[i:i + n, 0], got[torch.arange(i, i + n, device="cuda") % 251, 0])


def test_quantize_of_most_columns():
    """One row of 2^30 - 1 columns, and the columns of one of 2^28 + 3."""
    room(40)
    D = (1 << 30) - 1
    x = torch.arange(D, device="cuda", dtype=torch.int32).remainder_(1009).add_(1).to(BF)[None]
    o = ssm().quantize_fp8(x)
    for at in (0, 1 << 29, D - 127 - 128 * 7):        # (the last block is cut short)
        at = at // 128 * 128
        n = min(128 * 9, D - at)
        few = ssm().quantize_fp8(x[:, at:at + n].contiguous())
        assert torch.equal(o["q"][:, at:at + n].view(torch.uint8), few["q"][:, :n].view(torch.uint8))
        assert torch.equal(o["scale"][:, at // 128:at // 128 + few["scale"].shape[1]], few["scale"])
    assert o["q"].shape[1] == D + 1 and int(o["q"].view(torch.uint8)[0, D]) == 0
    del o
    x = x[:, :(1 << 28) + 3]
    o = ssm().quantize_fp8(x, rows=False, columns=True)
    for i in range(0, x.shape[1], 1 << 26):
        v = x[0, i:i + (1 << 26)].float()
        assert torch.equal(o["scale_t"][i:i + (1 << 26), 0], (v.double() / 448.0).float())
        assert bool((o["qt"][i:i + (1 << 26), 0].float() == 448.0).all())
    assert int(o["qt"].view(torch.uint8)[:, 1:].max()) == 0
