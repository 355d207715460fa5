"""The operators at a block's ends against 64 bits: quantisation to e4m3 with a scale for each block of 128, the residual's
addition with the norm (8-bit output, gradients), the product of 8-bit operands.

Tolerances count roundings: half a step of the output's type (bf16 2^-8, fp32 2^-24 relative; e4m3 half the distance of the
values around) once, and 2^-24 of the magnitudes that are added for every addition in a row.  u = 2^-24 below.
"""
import math

import pytest
import torch

import projection_ref as R

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
u = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: u}
LEAST_SCALE = torch.tensor(2.0 ** -100 / 448.0, dtype=F32)


def ssm():
    import selective_state_space_57_amd as m
    return m


class Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, *shape, scale=1.0, dtype=F32, wide=0):
        """A normal matrix; `wide`: its rows are parts of rows that are longer by so much."""
        v = torch.randn(*shape, generator=self.g, device="cuda") * scale
        if wide:
            base = torch.full((shape[0], shape[1] + wide), float("nan"), device="cuda").to(dtype)
            out = base[:, wide // 2:wide // 2 + shape[1]]
            out.copy_(v)
            return out
        return v.to(dtype)

    def codes(self, *shape):
        """Any e4m3 values but NaN, evenly."""
        c = torch.randint(0, 254, shape, generator=self.g, device="cuda")
        return (c + (c >= 127)).to(torch.uint8).view(F8)

    def scales(self, *shape):
        return torch.exp(torch.randn(*shape, generator=self.g, device="cuda"))


def inside(got, want, tol, what=""):
    """Every entry within its tolerance."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), "%s: %d off, the worst %.3g of its tolerance" % (what, int(bad.sum()), float((d / tol.clamp(min=1e-300)).max()))


def check_codes(q, scale, x, rows):
    """Scales are exact; codes are the nearest values (1 / scale and the product with it are rounded: 2 u of the value);
    behind the end of a row there are zeros."""
    T, D = x.shape
    assert q.shape == (T, R.up(D, 16)) and q.dtype == F8
    assert torch.equal(scale, R.scales(x, rows))
    v = x.double() / R.spread(scale.double(), rows, x.shape)
    inside(q[:, :D], v, R.half_step(v) + 4 * u * v.abs(), "codes")
    assert int(q.view(torch.uint8)[:, D:].count_nonzero()) == 0


# ---------------------------------------------------------------------------------------------------------------
# quantisation

SHAPES = [(1, 1), (1, 16), (3, 17), (2, 127), (16, 128), (128, 128), (129, 130), (127, 1000), (257, 2560), (1, 10576), (1999, 64)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", SHAPES)
def test_quantize(T, D, dtype):
    r = Rand(T * 7 + D)
    for wide in (0, 6):
        x = r(T, D, dtype=dtype, wide=wide) * torch.exp(2 * r(1, D)).to(dtype) if not wide else r(T, D, dtype=dtype, wide=wide)
        o = ssm().quantize_fp8(x)
        assert o["qt"] is None and o["scale_t"] is None
        check_codes(o["q"], o["scale"], x, 1)
        both = ssm().quantize_fp8(x, columns=True)
        assert torch.equal(both["q"].view(torch.uint8), o["q"].view(torch.uint8)) and torch.equal(both["scale"], o["scale"])
        check_codes(both["qt"], both["scale_t"], x.t(), 1)
        only = ssm().quantize_fp8(x, rows=False, columns=True)
        assert only["q"] is None and only["scale"] is None
        assert torch.equal(only["qt"].view(torch.uint8), both["qt"].view(torch.uint8)) and torch.equal(only["scale_t"], both["scale_t"])
        b = ssm().quantize_fp8_blocks(x, columns=True)
        check_codes(b["q"], b["scale"], x, 128)
        check_codes(b["qt"], b["scale_t"], x.t(), 128)
        assert torch.equal(b["q"].view(torch.uint8)[:, :D], b["qt"].view(torch.uint8)[:, :T].t())
        assert torch.equal(b["scale"], b["scale_t"].t())
        assert torch.equal(ssm().quantize_fp8_blocks(x)["q"].view(torch.uint8), b["q"].view(torch.uint8))


def test_quantize_many_rows():
    """More units of 512 columns than the plan for few takes, in rows that are not 16-byte aligned."""
    x = Rand(1)(20001, 77, dtype=BF)
    o = ssm().quantize_fp8(x)
    check_codes(o["q"], o["scale"], x, 1)
    x = Rand(2)(5001, 2560, dtype=BF, wide=2)
    o = ssm().quantize_fp8(x)
    check_codes(o["q"], o["scale"], x, 1)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_every_bf16(rows):
    """Every finite bf16 value, in blocks of ordinary ones: magnitudes from the smallest to the largest, zeros of both signs,
    blocks of nothing but zeros."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(BF)
    x = torch.where(bits.isfinite(), bits, torch.zeros((), dtype=BF, device="cuda")).view(512, 128).repeat(1, 2)
    x[:, 128:] = 0
    x[5, 130] = 3.0
    f = ssm().quantize_fp8 if rows == 1 else ssm().quantize_fp8_blocks
    o = f(x, columns=True)
    check_codes(o["q"], o["scale"], x, rows)
    check_codes(o["qt"], o["scale_t"], x.t(), rows)
    if rows == 1:
        assert torch.equal(o["scale"].min(), LEAST_SCALE.cuda())


def test_quantize_ties_and_top():
    """The largest entry of a block is 448 exactly; halves go to the even code."""
    x = torch.zeros(2, 128, device="cuda")
    x[0, 0], x[0, 1:6] = 448.0, torch.tensor([17.0, 19.0, -17.0, 21.0, 432.0], device="cuda")    # steps of 2 from 16, of 32 from 256
    x[1, 0], x[1, 1:4] = -448.0, torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9], device="cuda")
    o = ssm().quantize_fp8(x)
    assert o["scale"].flatten().tolist() == [1.0, 1.0]
    assert o["q"][0, :6].float().tolist() == [448.0, 16.0, 20.0, -16.0, 20.0, 448.0]
    assert o["q"][1, :4].float().tolist() == [-448.0, 0.0, 2.0 ** -8, 2.0 ** -9]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_not_finite(bad, dtype):
    """What is not finite stays in its block, which has a NaN scale, or an infinite one: no value of it (nor the zeros that
    fill up its last 16) is a number."""
    x = Rand(3)(200, 300, dtype=dtype)
    x[130, 140] = bad
    clean = x.clone()
    clean[130, 140] = 0
    o, c = ssm().quantize_fp8(x, columns=True), ssm().quantize_fp8(clean, columns=True)
    for k, s, at in (("q", "scale", (130, slice(128, 256))), ("qt", "scale_t", (140, slice(128, 208)))):
        got = R.values(o[k], o[s], 1)
        assert got[at].isnan().all()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[at] = False
        assert torch.equal(got[keep], R.values(c[k], c[s], 1)[keep])
    assert int(o["qt"].view(torch.uint8)[:, 200:].count_nonzero()) == 0
    assert int(o["q"].view(torch.uint8)[:, 300:].count_nonzero()) == 0
    b = ssm().quantize_fp8_blocks(x, columns=True)
    got = R.values(b["q"], b["scale"], 128)
    assert got[128:, 128:256].isnan().all() and got[:128].isfinite().all() and got[:, 256:].isfinite().all()
    assert int(b["qt"].view(torch.uint8)[:, 200:].count_nonzero()) == 0


def test_quantize_into_given():
    """Outputs that are parts of wider rows are written there, and nothing beside them."""
    x = Rand(4)(70, 200, dtype=BF)
    want = ssm().quantize_fp8(x, columns=True)
    base = {k: torch.full((v.shape[0] + 1, v.shape[1] + (32 if v.dtype == F8 else 3)), 0.5, device="cuda").to(v.dtype) for k, v in want.items()}
    given = {k: base[k][:v.shape[0], :v.shape[1]] for k, v in want.items()}
    got = ssm().quantize_fp8(x, columns=True, **given)
    for k, v in want.items():
        assert got[k] is given[k]
        assert torch.equal(got[k].float(), v.float())
        assert (base[k][-1].float() == 0.5).all() and (base[k][:, v.shape[1]:].float() == 0.5).all()


# ---------------------------------------------------------------------------------------------------------------
# norm

DIMS = [(1, 1), (3, 7), (5, 64), (1, 768), (9, 511), (33, 1000), (7, 1544), (130, 2560), (3, 2561), (2, 4096), (5, 5120), (3, 8190), (2, 16384), (2, 16383)]


def additions(D):
    """Additions in a row at most: a lane's, over a wave, over 16 waves; and those of eps, mean, root, reciprocal, products."""
    return 64 + 6 + 16 + 8


@pytest.mark.parametrize("res", [None, BF, F32], ids=["none", "bf16", "f32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["x16", "x32"])
@pytest.mark.parametrize("T,D", DIMS)
def test_add_norm(T, D, dtype, res):
    r = Rand(T + 31 * D)
    x, w = r(T, D, dtype=dtype, wide=5), 1 + r(D, scale=0.2)
    residual = None if res is None else r(T, D, scale=2.0, dtype=res, wide=3)
    eps = 1e-5
    h, y = R.add_norm(x, residual, w, eps)
    got, kept, scale = ssm().add_norm_fwd(x, w, residual, eps=eps)
    assert got.dtype == dtype and scale is None
    tol = additions(D) * u * y.abs()
    inside(got, y, HALF[dtype] * y.abs() + tol, "y")
    if residual is None:
        assert kept is None
    else:
        assert kept.dtype == res
        inside(kept, h, (HALF[res] + u) * h.abs(), "h")
    q, kept8, scale = ssm().add_norm_fwd(x, w, residual, eps=eps, y_dtype=F8)
    assert q.shape == (T, R.up(D, 16)) and q.dtype == F8
    s = R.magnitudes(y, 1).clamp(min=R.LEAST) / R.TOP
    inside(scale, s, (additions(D) + 2) * u * s, "scale")
    v = y / R.spread(scale.double(), 1, y.shape)
    inside(q[:, :D], v, R.half_step(v) + (additions(D) + 4) * u * v.abs() * 2, "codes")
    assert int(q.view(torch.uint8)[:, D:].count_nonzero()) == 0
    assert (kept8 is None) == (kept is None) and (kept is None or torch.equal(kept8, kept))


@pytest.mark.parametrize("htype", [BF, F32], ids=["h16", "h32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["dy16", "dy32"])
@pytest.mark.parametrize("T,D", DIMS + [(2100, 200), (700, 2560)])
def test_add_norm_grads(T, D, dtype, htype):
    r = Rand(T + 17 * D)
    h, w, dy = r(T, D, scale=2.0, dtype=htype, wide=3), 1 + r(D, scale=0.2), r(T, D, dtype=dtype, wide=5)
    for dh in (None, r(T, D, dtype=htype)):
        ds, dw, size, dwsize = R.add_norm_grads(h, w, dy, dh, 1e-5)
        g = ssm().add_norm_bwd(h, w, dy, dh)
        assert g["dx"].dtype == dtype and g["dresidual"].dtype == htype and g["dweight"].dtype == F32
        for k in ("dx", "dresidual"):
            inside(g[k], ds, HALF[g[k].dtype] * ds.abs() + 2 * additions(D) * u * size, k)
        # a lane adds the rows of its turns, a workgroup its 4 teams, a second kernel the workgroups in 16 runs and those
        inside(g["dweight"], dw, (additions(D) + T / 4 + 4 + 512 / 16 + 16) * u * dwsize, "dweight")


def test_add_norm_gradient_against_differences():
    """The formula's gradient and a difference quotient of the 64-bit definition agree, so the kernel's does."""
    r = Rand(5)
    h, w, dy, dh = r(4, 40), 1 + r(40, scale=0.2), r(4, 40), r(4, 40)
    v, vw = r(4, 40).double(), r(40).double()

    def loss(e, ew):
        hh, y = R.add_norm(h.double() + e * v, None, w.double() + ew * vw, 1e-5)
        return (y * dy.double()).sum() + (hh * dh.double()).sum()
    g = ssm().add_norm_bwd(h, w, dy, dh)
    # differences of step 1e-5 in 64 bits are off by about 1e-10 (curvature) + 1e-11 (cancellation); the kernel's sums by 2^-20
    for k, d, got in (("h", (loss(1e-5, 0) - loss(-1e-5, 0)) / 2e-5, (g["dresidual"].double() * v).sum()),
                      ("w", (loss(0, 1e-5) - loss(0, -1e-5)) / 2e-5, (g["dweight"].double() * vw).sum())):
        assert abs(float(got - d)) <= 2.0 ** -18 * (4 * 40) ** 0.5 * 4, k


def test_add_norm_in_place():
    r = Rand(6)
    x, res, w = r(37, 2560, dtype=BF), r(37, 2560), 1 + r(2560, scale=0.1)
    y, h, _ = ssm().add_norm_fwd(x, w, res)
    res2, x2 = res.clone(), x.clone()
    y2, h2, _ = ssm().add_norm_fwd(x2, w, res2, residual_out=res2, y=x2)
    assert y2 is x2 and h2 is res2 and torch.equal(y2, y) and torch.equal(h2, h)
    y3, h3, _ = ssm().add_norm_fwd(x, w, residual_dtype=F32)          # the first block: x starts the residual stream
    assert h3.dtype == F32 and torch.equal(h3, x.float())
    assert torch.equal(y3, ssm().add_norm_fwd(x, w)[0])
    dy, dh = r(37, 2560, dtype=BF), r(37, 2560)
    g = ssm().add_norm_bwd(h, w, dy, dh)
    dy2, dh2 = dy.clone(), dh.clone()
    g2 = ssm().add_norm_bwd(h, w, dy2, dh2, dx=dy2, dresidual=dh2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k
    same = ssm().add_norm_bwd(h.to(BF), w, dy, dh.to(BF))
    assert same["dx"] is same["dresidual"]
    two = ssm().add_norm_bwd(h.to(BF), w, dy, dh.to(BF), dx=torch.empty_like(dy), dresidual=torch.empty_like(dy))
    assert torch.equal(two["dx"], same["dx"]) and torch.equal(two["dresidual"], same["dx"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_add_norm_not_finite(bad):
    """What is not finite reaches its own row only: NaN, in 8 bits as the scales' NaN or the codes'."""
    r = Rand(7)
    for D in (200, 1001, 2560):
        x, res, w = r(9, D, dtype=BF), r(9, D), 1 + r(D, scale=0.1)
        y0, h0, _ = ssm().add_norm_fwd(x, w, res)
        q0, _, s0 = ssm().add_norm_fwd(x, w, res, y_dtype=F8)
        x[4, 3] = bad
        y, h, _ = ssm().add_norm_fwd(x, w, res)
        q, _, s = ssm().add_norm_fwd(x, w, res, y_dtype=F8)
        rest = [i for i in range(9) if i != 4]
        assert torch.equal(y[rest], y0[rest]) and torch.equal(h[rest], h0[rest])
        assert torch.equal(q[rest].float(), q0[rest].float()) and torch.equal(s[rest], s0[rest])
        assert not y[4, 3].isfinite() and not R.values(q[4:5], s[4:5], 1)[0, 3].isfinite()
        if math.isnan(bad):
            assert y[4].isnan().all() and s[4].isnan().all()
        assert int(q.view(torch.uint8)[:, D:].count_nonzero()) == 0


def test_add_norm_rows_of_zeros():
    w = torch.ones(300, device="cuda")
    x = torch.zeros(5, 300, device="cuda", dtype=BF)
    q, _, s = ssm().add_norm_fwd(x, w, y_dtype=F8)
    assert int(q.view(torch.uint8).count_nonzero()) == 0 and (s == LEAST_SCALE.cuda()).all()
    g = ssm().add_norm_bwd(x, w, torch.ones_like(x))
    inside(g["dx"], torch.full((5, 300), 1e-5 ** -0.5, dtype=torch.float64, device="cuda"), torch.full((5, 300), 2.0 ** -7 * 317, dtype=torch.float64, device="cuda"))
    assert int(g["dweight"].count_nonzero()) == 0


# ---------------------------------------------------------------------------------------------------------------
# product

# what the 8-bit matrix instructions drop of a block's inner sum: below 2^-12 of the largest of their products, for each of
# the (at most 16) groups that an instruction adds up, measured; fp32 results use others and drop nothing.  Additions in a
# row: 128 of a block, the blocks and their scales, 8 waves'
DROPPED = 2.0 ** -12


def tolerance(a, sa, b, sb, b_rows, out, want, size):
    blocks = (a.shape[1] + 127) // 128
    tol = HALF[out] * want.abs() + 2 * (128 + 2 * blocks + 8 + 4) * u * size
    if out == BF:
        big_a = R.magnitudes(a, 1) * sa.double()
        big_b = R.magnitudes(b, b_rows) * sb.double()
        if b_rows > 1:
            big_b = big_b.repeat_interleave(b_rows, 0)[:b.shape[0]]
        tol = tol + 16 * DROPPED * big_a @ big_b.T
    return tol


MM = [(1, 1, 16), (1, 3352, 768), (3, 5, 48), (16, 16, 128), (17, 130, 144), (64, 80, 1040), (1, 200, 10576), (127, 129, 256),
      (128, 128, 128), (129, 257, 400), (200, 10576, 64), (300, 300, 2560), (513, 1000, 160), (1000, 70, 5120), (2100, 2600, 272)]


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("b_rows", [128, 1], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,N,K", MM)
def test_matmul(M, N, K, b_rows, out):
    r = Rand(M + 3 * N + 5 * K)
    blocks = (K + 127) // 128
    a, sa = r.codes(M, K), r.scales(M, blocks)
    b, sb = r.codes(N, K), r.scales(-(-N // b_rows), blocks)
    if b_rows == 1 and N == 1:
        b_rows = 128
    want, size = R.product(a, sa, b, sb, b_rows)
    got = ssm().matmul_fp8(a, sa, b, sb, out_dtype=out)
    assert got.dtype == out and got.shape == (M, N)
    inside(got, want, tolerance(a, sa, b, sb, b_rows, out, want, size), "out")
    if out == F32:   # rounding errors go either way: over many results they are far below their bound
        assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,b_rows", [(1, 150, 272, 128), (9, 33, 128, 1), (50, 260, 1168, 128), (150, 140, 400, 1), (520, 530, 272, 128), (33, 1025, 144, 1)])
def test_matmul_of_whole_numbers(M, N, K, b_rows, out):
    """Small whole numbers under scales that are powers of two: every product and sum is exact, and so is every result but
    for its one rounding."""
    r = Rand(M * N)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=r.g, device="cuda").float().to(F8)

    def powers(*shape):
        return torch.exp2(torch.randint(-2, 3, shape, generator=r.g, device="cuda").float())
    blocks = (K + 127) // 128
    a, sa, b, sb = whole(M, K), powers(M, blocks), whole(N, K), powers(-(-N // b_rows), blocks)
    want, _ = R.product(a, sa, b, sb, b_rows)
    assert torch.equal(ssm().matmul_fp8(a, sa, b, sb, out_dtype=out), want.to(out))


# Every plan of a launch: tiles of 256 rows, whole and with the last turn in halves, of 192 rows, of 128; cut columns and rows.
@pytest.mark.parametrize("M,N,K,b_rows,out", [
    (4100, 4001, 144, 128, BF), (4099, 2560, 400, 128, BF), (8191, 2561, 272, 128, BF), (16389, 10576, 144, 128, BF),
    (8192, 8193, 1040, 128, BF), (4099, 3001, 272, 1, BF), (4099, 3001, 272, 1, F32), (4099, 3001, 272, 128, F32), (2000, 2100, 272, 1, F32),
    (16000, 200, 272, 128, BF), (200, 20001, 272, 1, BF), (1030, 1000, 2064, 128, BF), (129, 4100, 1040, 128, F32)])
def test_matmul_plans(M, N, K, b_rows, out):
    """Small whole numbers under scales that are powers of two, so that fp32 products are exact; every element is checked."""
    r = Rand(M + N)
    blocks = (K + 127) // 128
    a = torch.randint(-3, 4, (M, K), generator=r.g, device="cuda").float().to(F8)
    b = torch.randint(-3, 4, (N, K), generator=r.g, device="cuda").float().to(F8)
    sa = torch.exp2(torch.randint(-2, 3, (M, blocks), generator=r.g, device="cuda").float())
    sb = torch.exp2(torch.randint(-2, 3, (-(-N // b_rows), blocks), generator=r.g, device="cuda").float())
    want = (a.float() * R.spread(sa, 1, a.shape)) @ (b.float() * R.spread(sb, b_rows, b.shape)).t()
    base = torch.full((M + 1, N + 2), 5.0, dtype=out, device="cuda")
    for _ in range(2):
        got = ssm().matmul_fp8(a, sa, b, sb, out=base[:M, :N])
        assert torch.equal(got, want.to(out))
    assert (base[M:] == 5.0).all() and (base[:, N:] == 5.0).all()


# Workgroups that share k: 16, 32 and 64 rows of a to one, and each width that n gives them (16, 32, 48, 64 and 96 rows of b);
# more blocks of k than waves, and fewer.
@pytest.mark.parametrize("out,b_rows", [(BF, 128), (BF, 1), (F32, 128), (F32, 1)], ids=["bf16-128", "bf16-1", "f32-128", "f32-1"])
@pytest.mark.parametrize("N", [2551, 5103, 10571, 16381, 24573])
@pytest.mark.parametrize("M,K", [(13, 1168), (29, 272), (61, 1168)])
def test_matmul_widths(M, N, K, out, b_rows):
    test_matmul_plans(M, N, K, b_rows, out)


@pytest.mark.parametrize("M,N,K,b_rows,out", [
    (127, 10571, 1168, 128, BF), (127, 10571, 272, 1, BF), (510, 2557, 2320, 128, BF), (510, 2557, 400, 128, F32), (250, 2557, 400, 1, F32),
    (640, 2560, 272, 128, BF), (767, 769, 4112, 1, F32), (4000, 100, 272, 128, BF), (20001, 61, 144, 1, BF)])
def test_matmul_few_tiles(M, N, K, b_rows, out):
    test_matmul_plans(M, N, K, b_rows, out)


# Tiles that have a CU to themselves: 64, 96 and 128 rows of b, and 256 of a; one block of k, fewer and more than the stages; cut rows and
# columns, rows of b under one scale that begin inside a tile.
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("K", [112, 144, 400, 1168])
@pytest.mark.parametrize("M,N", [(767, 2557), (730, 2560), (1000, 2555), (250, 10571), (1001, 4090), (129, 16001), (2001, 2550),
                                 (510, 10571)])
def test_matmul_single_turn(M, N, K, b_rows):
    test_matmul_plans(M, N, K, b_rows, BF)


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 37, 144), (30, 200, 272), (300, 400, 272)])
def test_matmul_strides(M, N, K, out):
    """Operands, scales and result as parts of wider rows: nothing beside them is used (NaN codes there) or written."""
    r = Rand(M + N + K)
    blocks = (K + 127) // 128
    a, sa, b, sb = r.codes(M, K), r.scales(M, blocks), r.codes(N, K), r.scales(-(-N // 128), blocks)

    def within(v, left, right, below):
        base = torch.full((v.shape[0] + below, left + v.shape[1] + right), 127, dtype=torch.uint8, device="cuda").view(F8) if v.dtype == F8 \
            else torch.full((v.shape[0] + below, left + v.shape[1] + right), float("nan"), dtype=v.dtype, device="cuda")
        base[:v.shape[0], left:left + v.shape[1]] = v
        return base[:v.shape[0], left:left + v.shape[1]]
    want = ssm().matmul_fp8(a, sa, b, sb, out_dtype=out)
    base = torch.full((M + 2, N + 9), 7.0, dtype=out, device="cuda")
    got = ssm().matmul_fp8(within(a, 16, 32, 1), within(sa, 1, 2, 1), within(b, 32, 16, 3), within(sb, 3, 0, 1), out=base[1:M + 1, 4:N + 4])
    assert torch.equal(got, want)
    base[1:M + 1, 4:N + 4] = 7.0
    assert (base == 7.0).all()


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 37, 144), (30, 200, 400), (300, 400, 272)])
def test_matmul_not_finite(M, N, K, out):
    """A NaN code or scale reaches its own row of the result (column, or columns under one scale), and nothing else."""
    r = Rand(M + N + K + 1)
    blocks = (K + 127) // 128
    a, sa, b, sb = r.codes(M, K), r.scales(M, blocks), r.codes(N, K), r.scales(N, blocks)
    clean = ssm().matmul_fp8(a, sa, b, sb, out_dtype=out)
    for what in ("a", "sa", "b", "sb", "inf"):
        t = {"a": a.clone(), "sa": sa.clone(), "b": b.clone(), "sb": sb.clone()}
        i = M // 2 if what in ("a", "sa", "inf") else N // 3
        if what in ("a", "b"):
            t[what].view(torch.uint8)[i, K - 1] = 127
        elif what == "inf":
            t["sa"][i, 0] = float("inf")
        else:
            t[what][i, blocks - 1] = float("nan")
        got = ssm().matmul_fp8(t["a"], t["sa"], t["b"], t["sb"], out_dtype=out)
        hit = torch.zeros_like(got, dtype=torch.bool)
        if what in ("a", "sa", "inf"):
            hit[i] = True
        else:
            hit[:, i] = True
        assert not got[hit].isfinite().any(), what
        assert torch.equal(got[~hit], clean[~hit]), what


def test_matmul_range_of_scales():
    """Scales from 2^-60 to 2^60 whose products stay finite."""
    r = Rand(9)
    a, b = r.codes(40, 256), r.codes(50, 256)
    sa = torch.exp2(torch.randint(-60, 60, (40, 2), generator=r.g, device="cuda").float())
    sb = torch.exp2(torch.randint(-30, 30, (1, 2), generator=r.g, device="cuda").float())
    want, size = R.product(a, sa, b, sb, 128)
    inside(ssm().matmul_fp8(a, sa, b, sb, out_dtype=F32), want, tolerance(a, sa, b, sb, 128, F32, want, size))


# The same for tiles: with a CU to themselves (64, 96 and 128 rows of b, 256 of a), of 128, 192 and 256 rows.
TILES = [(767, 2557, 272, BF), (250, 10571, 144, BF), (1001, 4090, 272, BF), (2001, 2550, 400, BF), (2750, 2560, 144, BF),
         (4099, 2560, 272, BF), (5100, 5120, 144, BF), (2100, 2600, 272, F32)]


@pytest.mark.parametrize("M,N,K,out", TILES)
def test_matmul_strides_of_tiles(M, N, K, out):
    test_matmul_strides(M, N, K, out)


@pytest.mark.parametrize("M,N,K,out", TILES)
def test_matmul_not_finite_of_tiles(M, N, K, out):
    test_matmul_not_finite(M, N, K, out)


@pytest.mark.parametrize("b_rows", [128, 1], ids=["blocks", "rows"])
@pytest.mark.parametrize("M,N,K,out", TILES)
def test_matmul_of_tiles(M, N, K, out, b_rows):
    test_matmul(M, N, K, b_rows, out)
