"""The packed Mamba-2 block operators on the GPU against their 64-bit definitions (packed_ref.py) on the same rounded
inputs: prompts, single tokens and gradients, at the lengths, sizes, strides and states where they can go wrong.

Tolerances.  A rounding is off by at most half a step: 2^-8 of the value in bf16, 2^-24 in fp32.
 - near(): norms of differences.  Independent roundings add up like squares, so an output behind k roundings of relative
   size r is within k r of the reference in the 2-norm, whatever the sizes of its terms.
 - within(): element by element, against the sum of the magnitudes of an output's terms, which bounds what roundings of
   the terms can do.
"""
import numpy as np
import pytest

import packed_ref as R

pytestmark = pytest.mark.gpu

BF, HALF32 = 2.0 ** -8, 2.0 ** -24


def T():
    import torch
    assert torch.cuda.is_available(), "GPU test run without a visible GPU"
    return torch


def ssm():
    import selective_state_space_57_amd as m
    return m


def f64(t):
    return None if t is None else t.detach().to("cpu").double()


def near(got, ref, tol, what=""):
    d, n = float((f64(got) - ref).norm()), float(ref.norm())
    print("%s: 2-norm %.2e of %.2e (allowed %.2e)" % (what, d / max(n, 1e-300), 1.0, tol), flush=True)
    assert d <= tol * n + 1e-30, (what, d, n, tol)


def within(got, bound, ref, what=""):
    worst = float(((f64(got) - ref).abs() - bound).max())
    assert worst <= 0, (what, worst)


class Rand:
    def __init__(self, seed):
        self.torch = T()
        self.g = self.torch.Generator().manual_seed(seed)

    def __call__(self, *shape, scale=1.0, dtype=None):
        t = self.torch.randn(*shape, generator=self.g) * scale
        return t.to(dtype or self.torch.float32).cuda()

    def wide(self, rows, cols, extra, dtype, at=0):
        """(rows, cols) cut out of wider rows."""
        return self(rows, cols + extra, dtype=dtype)[:, at:at + cols]


def packed(lens, lead=0, tail=0):
    """cu_seqlens on the device and as a list, and the number of rows."""
    torch = T()
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32).cuda(), cu, cu[-1] + tail


def states(r, S, tail, mode):
    """(state, state_idx, has_state) of a mode: none, plain, slots (permuted, one index outside), some (has_state)."""
    torch = T()
    if mode == "none":
        return None, None, None
    if mode == "plain":
        return r(S, *tail), None, None
    idx = torch.randperm(S + 2, generator=r.g)[:S].to(torch.int32)
    if S > 2:
        idx[1], idx[2] = -1, S + 2
    has = (torch.arange(S) % 2 == 0).cuda() if mode == "some" else None
    return r(S + 2, *tail), idx.cuda(), has


def last_pool(pool, idx, last):
    """What the pool holds after the call."""
    out = f64(pool).clone()
    for s in range(last.shape[0]):
        k = s if idx is None else int(idx[s])
        if 0 <= k < out.shape[0]:
            out[k] = last[s]
    return out


# ---------------------------------------------------------------------------------------------------------------
# convolution

CONV = [
    # lens, channels, width, dtype, extra columns, states, activation, rows before / behind the sequences
    ([1], 8, 4, "bf16", 0, "plain", True, 0, 0),
    ([5, 0, 1, 2, 3, 40], 24, 4, "bf16", 8, "some", True, 0, 3),
    ([3, 64, 129, 0], 2056, 4, "bf16", 0, "slots", True, 2, 5),
    ([70, 9, 300], 40, 3, "f32", 4, "slots", True, 0, 0),
    ([33, 1, 0, 2], 7, 2, "f32", 0, "plain", False, 0, 1),
    ([17, 4], 13, 4, "bf16", 3, "some", True, 1, 0),
    ([8, 8, 8], 16, 1, "bf16", 0, "none", True, 0, 0),
    ([1000], 520, 4, "bf16", 8, "none", False, 0, 0),
    ([2] * 70, 12, 4, "f32", 0, "some", True, 0, 0),
]


def conv_case(k):
    torch = T()
    lens, D, K, dtype, extra, mode, act, lead, tail = CONV[k]
    r = Rand(100 + k)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cu, cul, rows = packed(lens, lead, tail)
    x = r.wide(rows, D, extra, dt, at=extra // 2)
    w, b = r(D, K, scale=0.5), r(D, scale=0.2)
    state, idx, has = states(r, len(lens), (D, K - 1), mode)
    first = R.first_states(len(lens), (D, K - 1), state, idx, has)
    return torch, lens, D, K, dt, act, r, cu, cul, rows, x, w, b, state, idx, has, first


def conv_bound(dt, u, x, w, b, first, cul, act):
    # fp32: K fused multiply-adds of magnitudes |w||x| (2^-24 each), then silu, whose hardware exponential and reciprocal
    # are good to 2^-22 and whose argument's rounding moves it by 2^-24 |pre| log2(e): 2^-20 of the sum of magnitudes
    # covers both for |pre| < 8; silu's slope is below 1.1
    _, mag, _ = R.conv(x.abs(), w.abs(), b.abs(), cul, first.abs(), False)
    return (BF if dt.itemsize == 2 else HALF32) * u.abs() + 2.0 ** -20 * mag + 1e-30


@pytest.mark.parametrize("k", range(len(CONV)))
def test_conv_packed(k):
    torch, lens, D, K, dt, act, r, cu, cul, rows, x, w, b, state, idx, has, first = conv_case(k)
    _, ref, last = R.conv(f64(x), f64(w), f64(b), cul, first, act)
    u = torch.full((rows, D + 8), 7.0, dtype=dt, device="cuda")[:, :D]
    out = None if state is None else torch.full_like(state, 3.0)
    got = ssm().conv1d_packed_fwd(x, w, cu, b, state=state, state_out=out, state_idx=idx, has_state=has, activation=act,
                                  u=u)
    torch.cuda.synchronize()
    assert got is u
    inside = slice(cul[0], cul[-1])
    within(u[inside], conv_bound(dt, ref, f64(x), f64(w), f64(b), first, cul, act)[inside], ref[inside], "u")
    assert bool((u[:cul[0]] == 7).all()) and bool((u[cul[-1]:] == 7).all())
    if state is not None:
        # windows are copies of inputs: exact, and the other slots untouched
        assert torch.equal(f64(out), last_pool(torch.full_like(state, 3.0), idx, last))
        pool = state.clone()
        ssm().conv1d_packed_fwd(x, w, cu, b, state=pool, state_out=pool, state_idx=idx, has_state=has, activation=act,
                                u=u)
        assert torch.equal(f64(pool), last_pool(state, idx, last))
        assert torch.equal(u, got)


@pytest.mark.parametrize("D,K,dtype,rows,extra", [(8, 4, "bf16", 1, 0), (2056, 4, "bf16", 33, 8), (13, 3, "bf16", 5, 1),
                                                  (44, 2, "f32", 7, 4), (9, 4, "f32", 3, 0), (16, 1, "bf16", 2, 0)])
def test_conv_step(D, K, dtype, rows, extra):
    torch = T()
    r = Rand(D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, w, b = r.wide(rows, D, extra, dt), r(D, K, scale=0.5), r(D, scale=0.2)
    idx = torch.randperm(rows + 2, generator=r.g)[:rows].to(torch.int32)
    if rows > 2:
        idx[0] = -1
    pool = r(rows + 2, D, K - 1)
    cul = list(range(rows + 1))
    first = R.first_states(rows, (D, K - 1), pool, idx, None)
    _, ref, last = R.conv(f64(x), f64(w), f64(b), cul, first)
    before = pool.clone()
    u = ssm().conv1d_slot_update(pool, x, w, b, state_idx=idx.cuda())
    torch.cuda.synchronize()
    within(u, conv_bound(dt, ref, f64(x), f64(w), f64(b), first, cul, True), ref, "u")
    assert torch.equal(f64(pool), last_pool(before, idx, last))


@pytest.mark.parametrize("k", range(len(CONV)))
def test_conv_packed_bwd(k):
    torch, lens, D, K, dt, act, r, cu, cul, rows, x, w, b, state, idx, has, first = conv_case(k)
    du = r.wide(rows, D, 8, dt)
    dl = r(len(lens), D, K - 1)
    dx = torch.full((rows, D + 16), 7.0, dtype=dt, device="cuda")[:, 8:8 + D]
    got = ssm().conv1d_packed_bwd(x, w, du, cu, b, state=state, state_idx=idx, has_state=has, dstate_out=dl,
                                  activation=act, want_dstate=True, dx=dx)
    torch.cuda.synchronize()
    ref = R.conv_grads(f64(x), f64(w), f64(b), cul, first, f64(du), f64(dl), act)
    inside = slice(cul[0], cul[-1])
    # dpre carries the slope's error (as silu's above, 2^-20), a few more fp32 roundings on the way
    small = 2.0 ** -19
    near(dx[inside], ref["dx"][inside], (BF if dt.itemsize == 2 else 0) + small, "dx")
    near(got["dweight"], ref["dweight"], small, "dweight")
    near(got["dbias"], ref["dbias"], small, "dbias")
    if K > 1:
        near(got["dstate"], ref["dstate"], small, "dstate")
    assert bool((dx[:cul[0]] == 7).all()) and bool((dx[cul[-1]:] == 7).all())
    again = ssm().conv1d_packed_bwd(x, w, du, cu, b, state=state, state_idx=idx, has_state=has, dstate_out=dl,
                                    activation=act, want_dstate=True)
    assert all(torch.equal(got[n], again[n]) for n in ("dweight", "dbias", "dstate"))


# ---------------------------------------------------------------------------------------------------------------
# norm

NORM = [
    # rows, dim, groups, dtype, gate (None, first, behind), center, bias, extra columns
    (1, 8, 1, "bf16", "first", False, False, 0),
    (3, 5, 5, "f32", "behind", False, True, 0),
    (7, 1536, 1, "bf16", "first", False, False, 8),
    (9, 1536, 8, "f32", "behind", True, True, 4),
    (5, 5120, 1, "bf16", "first", False, True, 0),
    (37, 5120, 8, "bf16", "behind", True, False, 16),
    (4, 16384, 1, "bf16", "first", True, True, 0),
    (3, 16384, 1, "f32", None, False, True, 0),
    (2, 16383, 1, "bf16", "first", False, False, 0),
    (6, 2 * 333, 2, "bf16", None, True, True, 1),
    (70, 130, 1, "bf16", "first", False, False, 3),
    (2000, 64, 2, "f32", "first", False, False, 0),
    (5, 7000, 1, "f32", "behind", False, True, 0),
    (3, 6000, 1, "bf16", "first", False, False, 0),
    (11, 3 * 1000, 3, "f32", "first", True, False, 0),
    (8, 260, 1, "f32", "first", False, False, 1),
]


def norm_case(k):
    torch = T()
    rows, D, G, dtype, gate, center, bias, extra = NORM[k]
    r = Rand(200 + k)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = r.wide(rows, D, extra, dt)
    if center:
        x += 0.5
    z = r.wide(rows, D, extra, dt) if gate else None
    w = 1 + r(D, scale=0.2)
    b = r(D, scale=0.3) if bias else None
    return torch, rows, D, G, dt, gate == "first", center, r, x, z, w, b


@pytest.mark.parametrize("k", range(len(NORM)))
def test_norm(k):
    torch, rows, D, G, dt, first, center, r, x, z, w, b = norm_case(k)
    y = ssm().gated_norm_fwd(x, w, b, z, groups=G, eps=1e-5, gate_first=first, center=center)
    torch.cuda.synchronize()
    ref = R.norm(f64(x), f64(w), f64(b), f64(z), G, 1e-5, first, center)
    # a sum over a lane's chunks and the team's lanes rounds at most 80 times; the gate's silu is good to 2^-20
    tol = (BF if dt.itemsize == 2 else 0) + 2.0 ** -18
    near(y, ref, tol, "y")
    within(y, tol * (ref.abs() + f64(w).abs() + (0 if b is None else f64(b).abs())), ref, "y")
    own = x.clone() if x.is_contiguous() else x
    got = ssm().gated_norm_fwd(own, w, b, z, groups=G, gate_first=first, center=center, y=own)
    assert got is own and torch.equal(own, y)


@pytest.mark.parametrize("k", range(len(NORM)))
def test_norm_bwd(k):
    torch, rows, D, G, dt, first, center, r, x, z, w, b = norm_case(k)
    dy = r.wide(rows, D, 8, dt)
    got = ssm().gated_norm_bwd(x, w, dy, b, z, groups=G, eps=1e-5, gate_first=first, center=center)
    torch.cuda.synchronize()
    ref = R.norm_grads(f64(x), f64(w), f64(b), f64(z), G, 1e-5, first, center, f64(dy))
    # dn - nh mean(dn nh) takes away what the norm cannot see: a group of n keeps at least about 1 - 2/n of it (none for
    # n = 1, where dx is nothing but the rest behind eps), so roundings (2^-18 as above) grow by n / (n - 2) in general;
    # groups of one or two channels are left to the element bound below
    n = D // G
    tol = (BF if dt.itemsize == 2 else 0) + 2.0 ** -17
    if n > 4:
        near(got["dx"], ref["dx"], tol, "dx")
    if z is not None:
        near(got["dz"], ref["dz"], tol, "dz") if n > 4 or not first else None
    near(got["dweight"], ref["dweight"], 2.0 ** -17, "dweight")
    near(got["dbias"], ref["dbias"], 2.0 ** -17, "dbias")
    again = ssm().gated_norm_bwd(x, w, dy, b, z, groups=G, eps=1e-5, gate_first=first, center=center)
    assert all(torch.equal(got[k], again[k]) for k in got if got[k] is not None)
    into = ssm().gated_norm_bwd(x, w, dy, b, z, groups=G, gate_first=first, center=center, dx=dy,
                                dz=z if z is not None else None)
    assert torch.equal(into["dx"], got["dx"]) and (z is None or torch.equal(into["dz"], got["dz"]))


# ---------------------------------------------------------------------------------------------------------------
# scan

SSD = [
    # lens, heads, groups, dstate, states, zoh, softplus, bias, D, chunks per segment, extra columns, lead, tail
    ([1], 1, 1, 64, "none", False, True, True, True, 0, 0, 0, 0),
    ([64], 8, 1, 128, "plain", False, True, True, True, 0, 0, 0, 0),
    ([65, 0, 1, 63, 200], 3, 1, 128, "some", False, True, True, True, 0, 8, 0, 7),
    ([200, 3, 130], 20, 2, 64, "slots", True, True, False, False, 1, 0, 3, 0),
    ([400, 64, 0, 128], 5, 1, 128, "some", False, True, True, False, 2, 8, 0, 0),
    ([130, 70], 6, 3, 256, "slots", True, True, True, True, 1, 8, 1, 2),
    ([257], 9, 1, 256, "plain", False, True, True, True, 0, 0, 0, 0),
    ([90, 100], 4, 4, 64, "plain", False, False, False, True, 1, 0, 0, 0),
    ([3] * 70, 2, 1, 64, "some", False, True, True, True, 0, 0, 0, 0),
    ([1500, 40], 8, 1, 128, "slots", False, True, True, True, 0, 0, 0, 0),
]


def ssd_case(k):
    torch = T()
    lens, H, G, N, mode, zoh, softplus, bias, dskip, seg, extra, lead, tail = SSD[k]
    r = Rand(300 + k)
    cu, cul, rows = packed(lens, lead, tail)
    bf = torch.bfloat16
    wide = r(rows, H * 64 + 2 * G * N + extra, dtype=bf)
    c = dict(cu=cu, x=wide[:, :H * 64].unflatten(1, (H, 64)))
    c["B"] = wide[:, H * 64:H * 64 + G * N].unflatten(1, (G, N))
    c["C"] = wide[:, H * 64 + G * N:H * 64 + 2 * G * N].unflatten(1, (G, N))
    c["dt"] = r.wide(rows, H, 3, bf)
    if not softplus:
        c["dt"] = (c["dt"].float().abs() * 0.05).to(bf)
    c["A"] = -torch.exp(torch.rand(H, generator=r.g) * 2.7).cuda()
    if zoh:
        c["A"][0] = 0.0
    c["bias"] = (torch.rand(H, generator=r.g) * 3 - 5).cuda() if bias else None
    c["D"] = 1 + r(H, scale=0.1) if dskip else None
    state, idx, has = states(r, len(lens), (H, 64, N), mode)
    first = R.first_states(len(lens), (H, 64, N), state, idx, has)
    return torch, r, c, cul, rows, state, idx, has, first, dict(softplus=softplus, zoh=zoh), dict(
        disc=1 if zoh else 0, softplus=softplus, segment_chunks=seg)


def ssd_ref(c, cul, first, how):
    return R.ssd(f64(c["x"]), f64(c["dt"]), f64(c["A"]), f64(c["B"]), f64(c["C"]), f64(c["bias"]), f64(c["D"]), cul, first,
                 **how)


# y stands behind three roundings to bf16 (M, the state's copy, y itself); the state behind decays whose logarithms, up to
# 2^7 in a chunk, are summed in fp32 (2^-17), a few of them along a sequence, and far smaller roundings of its products
TOL_Y, TOL_STATE = 3 * BF, 2.0 ** -15


@pytest.mark.parametrize("k", range(len(SSD)))
def test_ssd_packed(k):
    torch, r, c, cul, rows, state, idx, has, first, how, kw = ssd_case(k)
    ref, last, mag = ssd_ref(c, cul, first, how)
    y = torch.full((rows, c["x"].shape[1], 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = None if state is None else torch.full_like(state, 3.0)
    args = (c["x"], c["dt"], c["A"], c["B"], c["C"], c["cu"], c["bias"], c["D"])
    got = ssm().ssd_packed_fwd(*args, state=state, state_out=out, state_idx=idx, has_state=has, y=y, **kw)
    torch.cuda.synchronize()
    assert got is y
    inside = slice(cul[0], cul[-1])
    near(y[inside], ref[inside], TOL_Y, "y")
    within(y[inside], (TOL_Y * mag + 1e-30)[inside], ref[inside], "y")
    assert bool((y[:cul[0]] == 7).all()) and bool((y[cul[-1]:] == 7).all())
    if state is not None:
        want = last_pool(torch.full_like(state, 3.0), idx, last)
        near(out, want, TOL_STATE, "state")
        pool = state.clone()
        y2 = ssm().ssd_packed_fwd(*args, state=pool, state_out=pool, state_idx=idx, has_state=has, **kw)
        assert torch.equal(y2[inside], y[inside])
        named = [s if idx is None else int(idx[s]) for s in range(first.shape[0])]
        named = [n for n in named if 0 <= n < state.shape[0]]
        assert torch.equal(pool[named], out[named])
        rest = [n for n in range(state.shape[0]) if n not in named]
        assert torch.equal(pool[rest], state[rest])


@pytest.mark.parametrize("H,G,N,rows,zoh", [(1, 1, 64, 1, False), (3, 1, 128, 5, False), (6, 2, 256, 4, True),
                                            (24, 1, 128, 33, False), (4, 4, 64, 3, True)])
def test_ssd_step(H, G, N, rows, zoh):
    torch = T()
    r = Rand(N + H)
    bf = torch.bfloat16
    x = r.wide(rows, H * 64, 1, bf).unflatten(1, (H, 64))     # rows of any alignment
    B, C = (r.wide(rows, G * N, 4, bf).unflatten(1, (G, N)) for _ in range(2))
    dt, A = r.wide(rows, H, 5, bf), -torch.exp(torch.rand(H, generator=r.g) * 2.7).cuda()
    if zoh:
        A[0] = 0.0
    bias, D = r(H) - 3, r(H)
    idx = torch.randperm(rows + 2, generator=r.g)[:rows].to(torch.int32)
    if rows > 2:
        idx[0], idx[2] = -1, rows + 2
    pool = r(rows + 2, H, 64, N)
    cul = list(range(rows + 1))
    first = R.first_states(rows, (H, 64, N), pool, idx, None)
    ref, last, mag = R.ssd(f64(x), f64(dt), f64(A), f64(B), f64(C), f64(bias), f64(D), cul, first, True, zoh)
    before = pool.clone()
    y = ssm().ssd_slot_update(pool, x, dt, A, B, C, bias, D, state_idx=idx.cuda(), disc=1 if zoh else 0)
    torch.cuda.synchronize()
    # fp32 throughout, N products a row: 2^-24 (N + 8) of the magnitudes at most, and y's own rounding
    within(y, BF * ref.abs() + HALF32 * (N + 64) * mag, ref, "y")
    near(pool, last_pool(before, idx, last), 2.0 ** -20, "state")
    named = [int(i) for i in idx if 0 <= int(i) < rows + 2]
    rest = [n for n in range(rows + 2) if n not in named]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("k", range(len(SSD)))
def test_ssd_packed_bwd(k):
    torch, r, c, cul, rows, state, idx, has, first, how, kw = ssd_case(k)
    H, G, N = c["x"].shape[1], c["B"].shape[1], c["B"].shape[2]
    dy = r.wide(rows, H * 64, 16, torch.bfloat16, at=8).unflatten(1, (H, 64))
    dl = r(len(cul) - 1, H, 64, N, scale=0.3)
    ref = R.ssd_grads(f64(c["x"]), f64(c["dt"]), f64(c["A"]), f64(c["B"]), f64(c["C"]), f64(c["bias"]), f64(c["D"]), cul,
                      first, f64(dy), f64(dl), **how)
    inside = slice(cul[0], cul[-1])
    # dx, dB, dC written side by side into wider rows, as the convolution's backward takes them
    wide = torch.full((rows, H * 64 + 2 * G * N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = {"dx": wide[:, :H * 64].unflatten(1, (H, 64)), "dB": wide[:, H * 64:H * 64 + G * N].unflatten(1, (G, N)),
           "dC": wide[:, H * 64 + G * N:H * 64 + 2 * G * N].unflatten(1, (G, N)),
           "ddt": torch.full((rows, H + 2), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:H + 1]}
    args = (c["x"], c["dt"], c["A"], c["B"], c["C"], dy, c["cu"], c["bias"], c["D"])
    got = ssm().ssd_packed_bwd(*args, state=state, state_idx=idx, has_state=has, dstate_out=dl, out=out, **kw)
    torch.cuda.synchronize()
    assert got["dx"] is out["dx"] and got["dB"] is out["dB"]
    # dx: M, G and dx itself are rounded to bf16; dB and dC: the head sum K and the outputs; ddt: itself, on fp32 sums.
    # The fp32 sums behind dA, ddt_bias, ddt: products (2^-16 at most) and the decays' logarithms (2^-17), a few of them
    # in every term: 2^-14
    near(got["dx"][inside], ref["dx"][inside], 3 * BF, "dx")
    near(got["dB"][inside], ref["dB"][inside], 3 * BF, "dB")
    near(got["dC"][inside], ref["dC"][inside], 3 * BF, "dC")
    near(got["ddt"][inside], ref["ddt"][inside], BF + 2.0 ** -14, "ddt")
    for n in ("dA", "ddt_bias", "dDskip"):
        near(got[n], ref[n], 2.0 ** -14, n)
    near(got["dstate"], ref["dstate"], TOL_STATE, "dstate")
    for t in (wide, out["ddt"]):
        assert bool((t[:cul[0]] == 7).all()) and bool((t[cul[-1]:] == 7).all())
    assert bool((wide[:, H * 64 + 2 * G * N:] == 7).all())
    again = ssm().ssd_packed_bwd(*args, state=state, state_idx=idx, has_state=has, dstate_out=dl, **kw)
    for n in got:
        a, b = (got[n], again[n]) if n in ("dA", "ddt_bias", "dDskip", "dstate") else (got[n][inside], again[n][inside])
        assert torch.equal(a, b), n
