"""What the packed SSD kernels keep of 32 bits: outputs in bf16 are the 64-bit values rounded once, and nothing else.

Every product on the matrix cores has one factor that is bf16 already and one in parts.  Two parts leave out 2^-16 of a
value at most, three 2^-24.  The decays' logarithms are summed without loss that counts, their exponentials are good to
2^-22 and the step sizes' to 2^-21; a sum of up to 512 terms in fp32 rounds by 2^-24 each, 2^-15 of the magnitudes at worst.
"""
import pytest

import packed_ref as R
from test_packed_gpu import BF, SSD, Rand, T, f64, near, packed, ssd_case, ssd_ref, ssm, within

pytestmark = pytest.mark.gpu

# what stands before the last rounding, of the sum of the magnitudes: 2^-16 (parts) + 2^-15 (sums) + 2^-19 (step, decay)
REST = 2.0 ** -14
# a decay below fp32's smallest normal number, 2^-126, is zero: what it multiplies, below 2^25 here, is lost up to 2^-101
TINY = 2.0 ** -100


@pytest.mark.parametrize("k", range(len(SSD)))
def test_y_is_rounded_once(k):
    torch, r, c, cul, rows, state, idx, has, first, how, kw = ssd_case(k)
    ref, _, mag = ssd_ref(c, cul, first, how)
    y = ssm().ssd_packed_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], c["cu"], c["bias"], c["D"], state=state,
                             state_idx=idx, has_state=has, **kw)
    torch.cuda.synchronize()
    inside = slice(cul[0], cul[-1])
    within(y[inside], (BF * ref.abs() + REST * mag + TINY)[inside], ref[inside], "y")


@pytest.mark.parametrize("k", range(len(SSD)))
def test_gradients_are_rounded_once(k):
    torch, r, c, cul, rows, state, idx, has, first, how, kw = ssd_case(k)
    H, N = c["x"].shape[1], c["B"].shape[2]
    dy = r(rows, H, 64, dtype=torch.bfloat16)
    dl = r(len(cul) - 1, H, 64, N, scale=0.3)
    wide = [f64(c[n]) for n in ("x", "dt", "A", "B", "C", "bias", "D")]
    ref = R.ssd_grads(*wide, cul, first, f64(dy), f64(dl), **how)
    # with every factor's magnitude the same formulas sum the magnitudes of the terms
    big = [t if t is None or n in "dt A bias" else t.abs() for n, t in zip(("x", "dt", "A", "B", "C", "bias", "D"), wide)]
    mag = R.ssd_grads(*big, cul, first.abs(), f64(dy).abs(), f64(dl).abs(), **how)
    got = ssm().ssd_packed_bwd(c["x"], c["dt"], c["A"], c["B"], c["C"], dy, c["cu"], c["bias"], c["D"], state=state,
                               state_idx=idx, has_state=has, dstate_out=dl, **kw)
    torch.cuda.synchronize()
    inside = slice(cul[0], cul[-1])
    for n in ("dx", "dB", "dC"):
        within(got[n][inside], (BF * ref[n].abs() + REST * mag[n] + TINY)[inside], ref[n][inside], n)


RESETS = [(64, False, (200, 500)), (128, False, (1000, 1e4)), (128, True, (200, 1e4)), (256, False, (20, 200, 1e4)),
          (64, True, (3, 10, 1000))]


def resetting(N, zoh, strong):
    """A quarter of the steps large, the others 1e-3 to 0.1."""
    torch = T()
    r = Rand(40 + N + zoh)
    H, lens = 4, [130, 64, 200, 3]
    cu, cul, rows = packed(lens)
    bf = torch.bfloat16
    x, dy = r(rows, H, 64, dtype=bf), r(rows, H, 64, dtype=bf)
    B, C = r(rows, 1, N, dtype=bf), r(rows, 1, N, dtype=bf)
    A = -torch.tensor([1.0, 8.0, 16.0, 12.0]).cuda()
    u = torch.rand(rows, H, generator=r.g) * 4.6 - 6.9                       # softplus: 1e-3 to 0.1
    big = torch.tensor(strong)[torch.randint(0, len(strong), (rows, H), generator=r.g)]
    dt = torch.where(torch.rand(rows, H, generator=r.g) < 0.25, big, u).to(bf).cuda()
    D = r(H)
    state, dl = r(len(lens), H, 64, N), r(len(lens), H, 64, N, scale=0.3)
    wide = [f64(t) for t in (x, dt, A, B, C)]
    mags = [wide[0].abs(), wide[1], wide[2], wide[3].abs(), wide[4].abs()]
    return torch, x, dt, A, B, C, D, dy, cu, cul, state, dl, wide, mags


# What decays between ordinary steps behind one that resets the state is as good as without it.

@pytest.mark.parametrize("N,zoh,strong", RESETS)
def test_y_behind_steps_that_reset_the_state(N, zoh, strong):
    torch, x, dt, A, B, C, D, dy, cu, cul, state, dl, wide, mags = resetting(N, zoh, strong)
    first = f64(state)
    ref, last, mag = R.ssd(*wide, None, f64(D), cul, first, True, zoh)
    out = torch.empty_like(state)
    y = ssm().ssd_packed_fwd(x, dt, A, B, C, cu, None, D, state=state, state_out=out, disc=int(zoh))
    torch.cuda.synchronize()
    within(y, BF * ref.abs() + REST * mag + TINY, ref, "y")
    # three parts; decays and sums as above, on the state's own magnitudes
    big = R.ssd(*mags, None, None, cul, first.abs(), True, zoh)[1]
    within(out, 2.0 ** -15 * big + TINY, last, "state")


@pytest.mark.parametrize("N,zoh,strong", RESETS)
def test_gradients_behind_steps_that_reset_the_state(N, zoh, strong):
    torch, x, dt, A, B, C, D, dy, cu, cul, state, dl, wide, mags = resetting(N, zoh, strong)
    first = f64(state)
    got = ssm().ssd_packed_bwd(x, dt, A, B, C, dy, cu, None, D, state=state, dstate_out=dl, disc=int(zoh))
    torch.cuda.synchronize()
    g = R.ssd_grads(*wide, None, f64(D), cul, first, f64(dy), f64(dl), True, zoh)
    gm = R.ssd_grads(*mags, None, f64(D).abs(), cul, first.abs(), f64(dy).abs(), f64(dl).abs(), True, zoh)
    mag = R.ssd(*wide, None, f64(D), cul, first, True, zoh)[2]
    for n in ("dx", "dB", "dC"):
        within(got[n], BF * g[n].abs() + REST * gm[n] + TINY, g[n], n)
    within(got["dstate"], 2.0 ** -15 * gm["dstate"] + TINY, g["dstate"], "dstate")
    # dl of a step is what sums over the steps of its chunk leave: of rows and columns of W, whose magnitudes are those of
    # |dy| |y| and |x| |dx|, about 16 roundings of 2^-24 each of twice the chunk's; nothing where the step's decay is 0
    om = (f64(dy).abs() * mag).sum(-1) + (f64(x).abs() * gm["dx"]).sum(-1)
    u, d, a, phi = R.steps(wide[1], None, wide[2], True, zoh)
    tol = torch.zeros_like(om)
    for b, e in zip(cul, cul[1:]):
        for t in range(b, e, 64):
            tol[t:min(t + 64, e)] = 2.0 ** -19 * om[t:min(t + 64, e)].sum(0)
    tol = torch.where(a > 2.0 ** -126, tol, torch.zeros_like(tol))
    dphi = (f64(x).abs() * (gm["dx"] - f64(D).abs()[:, None] * f64(dy).abs())).sum(-1) / phi
    slope = 1 / (1 + torch.exp(-u))
    ddt = (wide[2].abs() * tol + 2.0 ** -17 * dphi) * slope
    within(got["ddt"], BF * g["ddt"].abs() + 2 * ddt + TINY, g["ddt"], "ddt")
    by_a = (d * a - phi).abs() / wide[2].abs() * dphi if zoh else torch.zeros_like(d)
    within(got["dA"], (d * tol + 2.0 ** -17 * by_a).sum(0) + 2.0 ** -17 * gm["dA"].abs() + TINY, g["dA"], "dA")
    within(got["ddt_bias"], ddt.sum(0) + 2.0 ** -17 * g["ddt"].abs().sum(0) + TINY, g["ddt_bias"], "ddt_bias")


LOWEST = [float("-inf"), -3.3895313892515355e38]     # (the lowest of bf16)


def masked(N):
    """A batch with steps that are masked by their step size, and where they are."""
    torch = T()
    r = Rand(50 + N)
    H, lens = 3, [70, 1, 129]
    cu, cul, rows = packed(lens)
    bf = torch.bfloat16
    x, dy = r(rows, H, 64, dtype=bf), r(rows, H, 64, dtype=bf)
    B, C = r(rows, 1, N, dtype=bf), r(rows, 1, N, dtype=bf)
    dt, A, D = r(rows, H, dtype=bf), -torch.rand(H, generator=r.g).cuda() * 7 - 1, r(H)
    off = (torch.rand(rows, H, generator=r.g) < 0.3).cuda()
    off[70] = True
    state, dl = r(3, H, 64, N), r(3, H, 64, N, scale=0.3)
    return torch, x, dt, A, B, C, D, dy, cu, cul, state, dl, off


@pytest.mark.parametrize("low", LOWEST)
@pytest.mark.parametrize("N,zoh", [(64, False), (128, True), (256, False)])
def test_steps_masked_by_their_size(low, N, zoh):
    """softplus of -infinity and of the type's lowest value is 0: such a step leaves the state as it is, and has no gradient.
    -200 gives 0 as well, in ordinary arithmetic: all outputs are the same bits."""
    torch, x, dt, A, B, C, D, dy, cu, cul, state, dl, off = masked(N)
    res = []
    for v in (low, -200.0):
        d = torch.where(off, torch.full_like(dt, v), dt)
        out, pool = torch.empty_like(state), state.clone()
        y = ssm().ssd_packed_fwd(x, d, A, B, C, cu, None, D, state=state, state_out=out, disc=int(zoh))
        g = ssm().ssd_packed_bwd(x, d, A, B, C, dy, cu, None, D, state=state, dstate_out=dl, disc=int(zoh))
        s = ssm().ssd_slot_update(pool, x[:3], d[:3], A, B[:3], C[:3], None, D, disc=int(zoh))
        torch.cuda.synchronize()
        res.append(dict(g, y=y, out=out, s=s, pool=pool))
    for n, t in res[0].items():
        assert bool(t.isfinite().all()), n
        assert torch.equal(t, res[1][n]), n
    assert bool((res[0]["ddt"][off] == 0).all())
    assert torch.equal(res[0]["out"][1], state[1])        # one step, masked


@pytest.mark.parametrize("N", [64, 128])
def test_largest_steps_under_zero_order_hold(N):
    """A step of the type's largest value resets the state to -x B / A; nothing of it is infinite.  Steps of 1e4 do the same in
    ordinary arithmetic: all outputs are the same bits."""
    torch, x, dt, A, B, C, D, dy, cu, cul, state, dl, off = masked(N)
    res = []
    for v in (3.3895313892515355e38, 1e4):
        d = torch.where(off, torch.full_like(dt, v), dt)
        out, pool = torch.empty_like(state), state.clone()
        y = ssm().ssd_packed_fwd(x, d, A, B, C, cu, None, D, state=state, state_out=out, disc=1)
        g = ssm().ssd_packed_bwd(x, d, A, B, C, dy, cu, None, D, state=state, dstate_out=dl, disc=1)
        s = ssm().ssd_slot_update(pool, x[:3], d[:3], A, B[:3], C[:3], None, D, disc=1)
        torch.cuda.synchronize()
        res.append(dict(g, y=y, out=out, s=s, pool=pool))
    for n, t in res[0].items():
        assert bool(t.isfinite().all()), n
        assert torch.equal(t, res[1][n]), n


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("N,at", [(64, 5), (64, 17), (128, 31), (128, 32), (128, 47), (128, 63), (256, 40), (256, 90)])
def test_what_is_not_finite_reaches_nothing_earlier(N, at, value):
    """One entry of x reaches its own column from its step on; one of B, C or dt its own group or head, and no earlier step."""
    torch = T()
    r = Rand(60 + N + at)
    H = 3
    cu, cul, rows = packed([130, 64])
    bf = torch.bfloat16
    c = dict(x=r(rows, H, 64, dtype=bf), dt=r(rows, H, dtype=bf), B=r(rows, 1, N, dtype=bf), C=r(rows, 1, N, dtype=bf))
    A, bias, D = -torch.rand(H, generator=r.g).cuda() - 0.5, r(H) - 3, r(H)
    state = r(2, H, 64, N)

    def run(**kw):
        c2, out = dict(c, **kw), torch.empty_like(state)
        y = ssm().ssd_packed_fwd(c2["x"], c2["dt"], A, c2["B"], c2["C"], cu, bias, D, state=state, state_out=out)
        torch.cuda.synchronize()
        return y, out

    def spoil(name, *place):
        t = c[name].clone()
        t[(at,) + place] = value
        return {name: t}

    clean, end = run()
    others = torch.ones(H, 64, dtype=torch.bool)
    others[1, 37] = False
    y, out = run(**spoil("x", 1, 37))
    assert torch.equal(y[:at], clean[:at]) and torch.equal(y[130:], clean[130:])
    assert torch.equal(y[:, others], clean[:, others]) and torch.equal(out[:, others], end[:, others])
    assert not bool(y[at:130, 1, 37].isfinite().any()) and not bool(out[0, 1, 37].isfinite().any())
    for name, place in (("B", (0, 9)), ("C", (0, 9)), ("dt", (1,))):
        if name == "dt" and value == float("-inf"):
            continue                                            # (a masked step)
        y, out = run(**spoil(name, *place))
        assert torch.equal(y[:at], clean[:at]) and torch.equal(y[130:], clean[130:]), name
        assert not bool(y[at].isfinite().all()), name
        if name == "C":
            assert torch.equal(y[at + 1:], clean[at + 1:]) and torch.equal(out, end)
        if name == "dt":
            assert torch.equal(y[:, [0, 2]], clean[:, [0, 2]]) and torch.equal(out[:, [0, 2]], end[:, [0, 2]])


@pytest.mark.parametrize("H,G,N,zoh", [(24, 1, 128, False), (10, 2, 64, True), (6, 1, 256, False)])
def test_states_and_step_gradients_keep_32_bits(H, G, N, zoh):
    """A layer's step sizes (1e-3 to 0.1) and decays (A from -16 to -1).  States and their gradients are fp32 products in three
    parts (2^-24 left out) and decays good to 2^-22; independent roundings, fewer than four of 2^-22 behind every term: 2^-20 of
    the 2-norm.  dA, ddt_bias and dDskip are sums over tokens of terms behind about twice as many: 2^-19.  (Two parts would
    leave 2.4e-6 in the states, 2^-18.7.)"""
    torch = T()
    r = Rand(110 + N)
    lens = [300, 1, 170, 200]
    cu, cul, rows = packed(lens)
    bf = torch.bfloat16
    x, B, C = (R.silu(r(rows, *s)).to(bf) for s in ((H, 64), (G, N), (G, N)))
    dt, dy = r(rows, H, dtype=bf), r(rows, H, 64, dtype=bf)
    A = -torch.exp(torch.rand(H, generator=r.g) * 2.77).cuda()
    step = torch.exp(torch.rand(H, generator=r.g) * 4.6 - 6.9)
    bias, D = (step + torch.log(-torch.expm1(-step))).cuda(), 1 + r(H, scale=0.1)
    state, dl = r(4, H, 64, N, scale=0.3), r(4, H, 64, N, scale=0.3)
    out = torch.empty_like(state)
    ssm().ssd_packed_fwd(x, dt, A, B, C, cu, bias, D, state=state, state_out=out, disc=int(zoh))
    got = ssm().ssd_packed_bwd(x, dt, A, B, C, dy, cu, bias, D, state=state, dstate_out=dl, disc=int(zoh))
    torch.cuda.synchronize()
    wide = [t.double() for t in (x, dt, A, B, C, bias, D)]
    with torch.device("cuda"):
        last = R.ssd(*wide, cul, state.double(), True, zoh)[1].cpu()
        ref = {k: v.cpu() for k, v in R.ssd_grads(*wide, cul, state.double(), dy.double(), dl.double(), True, zoh).items()}
    near(out, last, 2.0 ** -21, "state")
    near(got["dstate"], ref["dstate"], 2.0 ** -20, "dstate")
    for n in ("dA", "ddt_bias", "dDskip"):
        near(got[n], ref[n], 2.0 ** -19, n)
