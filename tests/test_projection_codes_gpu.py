"""Codes of the 8-bit quantisation, bit for bit: the fp32 quotient of a value and its scale, rounded to the nearest e4m3 value
(halves to the even one).  The quotient in 64 bits, rounded to 32, is the correctly rounded one (53 bits are more than twice 24
and two), so nothing here has a tolerance.
"""
import pytest
import torch

import projection_ref as R
from test_projection_gpu import BF, F32, F8, Rand, ssm

pytestmark = pytest.mark.gpu


def codes_of(x, scale, rows):
    """The code of every entry, on the CPU."""
    v = x.double().cpu() / R.spread(scale.double().cpu(), rows, x.shape)
    return v.float().to(F8).view(torch.uint8)


def same_codes(q, scale, x, rows, what):
    T, D = x.shape
    assert torch.equal(scale, R.scales(x, rows)), what
    got, want = q.view(torch.uint8)[:, :D].cpu(), codes_of(x, scale, rows)
    bad = got != want
    assert not bad.any(), "%s: %d of %d codes are not the nearest to their quotient" % (what, int(bad.sum()), bad.numel())


def every_form(x):
    o = ssm().quantize_fp8(x)
    same_codes(o["q"], o["scale"], x, 1, "rows alone")
    o = ssm().quantize_fp8(x, columns=True)
    same_codes(o["q"], o["scale"], x, 1, "rows")
    same_codes(o["qt"], o["scale_t"], x.t(), 1, "columns")
    o = ssm().quantize_fp8_blocks(x, columns=True)
    same_codes(o["q"], o["scale"], x, 128, "blocks")
    same_codes(o["qt"], o["scale_t"], x.t(), 128, "blocks of the transposed matrix")


def borders(r, T, D, lo=-30, hi=30):
    """fp32 rows whose values lie at the borders between codes, a unit in the last place beside them and two: of each block of
    128 the first is the largest, of any mantissa and of magnitudes 2^lo to 2^hi."""
    top = torch.exp2(lo + (hi - lo) * torch.rand(T, R.up(D, 128) // 128, generator=r.g, device="cuda")).repeat_interleave(128, 1)[:, :D]
    scale = (top.double() / R.TOP).float().double()
    k = 2 * torch.randint(0, 16, (T, D), generator=r.g, device="cuda") + 1
    up = torch.randint(0, 15, (T, D), generator=r.g, device="cuda")
    tie = k * torch.exp2(-10.0 + torch.where(k > 15, up, torch.zeros_like(up)).double())
    v = (scale * tie).float()
    near = (v.view(torch.int32) + torch.randint(-2, 3, (T, D), generator=r.g, device="cuda").int()).view(F32)
    sign = 1 - 2 * torch.randint(0, 2, (T, D), generator=r.g, device="cuda")
    x = torch.where((tie < 440) & (near > 0), near, v * 0) * sign
    x[:, ::128] = top[:, ::128]
    return x


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(257, 1000), (1, 5120), (300, 2560)])
def test_codes(T, D, dtype):
    r = Rand(T + D)
    every_form((r(T, D) * torch.exp(r(1, D))).to(dtype))


@pytest.mark.parametrize("lo,hi", [(-30, 30), (-99, -80), (-85, -60), (100, 126)])
def test_codes_at_their_borders(lo, hi):
    x = borders(Rand(hi - lo), 300, 640, lo, hi)
    o = ssm().quantize_fp8(x)
    same_codes(o["q"], o["scale"], x, 1, "rows alone")
    o = ssm().quantize_fp8(x.t().contiguous(), columns=True)
    same_codes(o["qt"], o["scale_t"], x, 1, "columns")
    every_form(x)


def test_codes_of_blocks_at_their_borders():
    """Blocks of 128 rows and columns, one largest magnitude in each: borders of its scale all over it."""
    r = Rand(4)
    x = borders(r, 1, 128 * 300).view(300, 128)
    x = x.repeat_interleave(128, 0)[:, torch.randperm(128, generator=r.g, device="cuda")]
    o = ssm().quantize_fp8_blocks(x, columns=True)
    same_codes(o["q"], o["scale"], x, 128, "blocks")
    same_codes(o["qt"], o["scale_t"], x.t(), 128, "blocks of the transposed matrix")


def test_codes_of_every_bf16():
    """Every finite bf16 value in blocks of other ones, zeros of both signs among them."""
    r = Rand(5)
    bits = torch.randperm(1 << 16, generator=r.g, device="cuda").to(torch.int32).to(torch.int16).view(BF)
    x = torch.where(bits.isfinite(), bits, torch.zeros((), dtype=BF, device="cuda")).view(512, 128)
    every_form(x)
    # and of one binade and the ones below it, where neighbours matter
    every_form(torch.where(x.abs() < 4, x, x.sign()).repeat(1, 3))


# One team of a wave, of four and of sixteen; rows that are no multiple of eight channels.
@pytest.mark.parametrize("D", [4, 128, 512, 1024, 2048, 8192, 16384])
def test_codes_of_the_norm(D):
    """Rows of ones of either sign, eps = 0 and a power of two of channels: the norm is 1 exactly and y is the weight, whose
    codes are those of a quantised matrix."""
    r = Rand(D)
    for seed in range(8):
        w = borders(r, 1, D).flatten() if seed % 2 else r(D).to(BF).float()
        x = (1 - 2 * torch.randint(0, 2, (5, D), generator=r.g, device="cuda")).to(BF)
        q, _, s = ssm().add_norm_fwd(x, w, eps=0.0, y_dtype=F8)
        same_codes(q, s, x.float() * w, 1, "norm")
