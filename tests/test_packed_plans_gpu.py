"""The launch plans that large batches get, on batches as small as still get them: several heads of a group one after the
other in the backward's main pass, segments where the sequences alone fill the card, long tiles of the convolution, and a
norm's workgroups that walk down several rows.  Each plan is computed here from the library's rule and asserted, and every
output compared with its 64-bit definition (packed_ref.py, run on the GPU).

Tolerances: test_packed_precision_gpu.py's for the scan, test_packed_gpu.py's for the others.
"""
import ctypes

import pytest

import packed_ref as R
from test_packed_gpu import BF, HALF32, Rand, T, near, packed, ssm, within
from test_packed_precision_gpu import REST, TINY

pytestmark = pytest.mark.gpu


def up(a, b):
    return -(-a // b)


def scan_plan(tokens, seqs, heads, groups, N):
    """(64-step chunks per segment, workgroups per segment, whether the sequences alone take more than half of the places)"""
    blocks = groups * up(heads // groups, 4)
    places = 256 if N == 256 else 512
    work, ends = (tokens // 64 + seqs // 2 + 1) * blocks, seqs * blocks // 2
    full = 2 * ends > places
    cps = up(2 * work, places) if full else up(work, places - ends)
    return min(max(cps, 4), up(tokens, 64)), blocks, full


def backward_plan(tokens, seqs, heads, groups):
    """(splits of a group's heads, heads of one)"""
    numbers, per = seqs + tokens // 64 + 1, heads // groups
    splits = min(up(2048, numbers * groups), per)
    hps = up(per, splits)
    return up(per, hps), hps


def check_workspaces(tokens, seqs, heads, groups, N):
    """The library's workspaces have the sizes that these plans ask for."""
    cps = scan_plan(tokens, seqs, heads, groups, N)[0]
    splits, _ = backward_plan(tokens, seqs, heads, groups)
    numbers, places = seqs + tokens // 64 + 1, 2 * (tokens // (cps * 64)) if up(tokens, 64) > cps else 0
    state, a = heads * 64 * N * 4, ssm()._abi
    walk = up(places * state, 256) * 256 + up(places * heads * 4, 256) * 256
    total = 2 * (up(numbers * state, 256) * 256 + walk + up(splits * tokens * groups * N * 4, 256) * 256)
    total += up(numbers * heads * 16, 256) * 256
    p = a.SsdPackedParams(ntokens=tokens, nseqs=seqs, nheads=heads, headdim=64, ngroups=groups, dstate=N, nslots=seqs,
                          io_dtype=a.SSM_BF16, dt_softplus=1)
    assert a.lib().ssm_ssd_packed_fwd_workspace_bytes(ctypes.byref(p)) == walk
    assert a.lib().ssm_ssd_packed_bwd_workspace_bytes(ctypes.byref(p)) == total


def scan_inputs(seed, lens, H, G, N):
    torch = T()
    r = Rand(seed)
    cu, cul, rows = packed(lens)
    bf = torch.bfloat16
    c = dict(x=r(rows, H, 64, dtype=bf), dt=r(rows, H, dtype=bf), B=r(rows, G, N, dtype=bf), C=r(rows, G, N, dtype=bf),
             dy=r(rows, H, 64, dtype=bf), A=-torch.exp(torch.rand(H, generator=r.g) * 2.7).cuda(),
             bias=(torch.rand(H, generator=r.g) * 3 - 5).cuda(), D=1 + r(H, scale=0.1),
             state=r(len(lens), H, 64, N), dl=r(len(lens), H, 64, N, scale=0.3))
    wide = {k: v.double() for k, v in c.items()}
    mags = {k: v if k in ("dt", "A", "bias") else v.abs() for k, v in wide.items()}
    return torch, c, cu, cul, wide, mags


def on_gpu(f, *args, **kw):
    with T().device("cuda"):
        out = f(*args, **kw)
    return {k: v.cpu() for k, v in out.items()} if isinstance(out, dict) else [v.cpu() for v in out]


@pytest.mark.parametrize("N,H,G,lens,zoh", [
    (64, 11, 1, [1] * 470 + [70, 130, 64, 65], False),
    (128, 11, 1, [130, 1, 64] + [1, 2] * 240 + [65, 200], True),
    (256, 7, 1, [1] * 640 + [100, 65], False),
    (128, 20, 2, [1] * 300 + [129, 63], False),
])
def test_backward_over_several_heads(N, H, G, lens, zoh):
    torch, c, cu, cul, w, m = scan_inputs(70 + N + H, lens, H, G, N)
    splits, hps = backward_plan(cul[-1], len(lens), H, G)
    check_workspaces(cul[-1], len(lens), H, G, N)
    assert hps >= 2 and splits * hps > H // G, (splits, hps)         # several heads, and a last split of fewer
    got = ssm().ssd_packed_bwd(c["x"], c["dt"], c["A"], c["B"], c["C"], c["dy"], cu, c["bias"], c["D"], state=c["state"],
                               dstate_out=c["dl"], disc=int(zoh))
    torch.cuda.synchronize()
    ref, mag = (on_gpu(R.ssd_grads, *(t[k] for k in ("x", "dt", "A", "B", "C", "bias", "D")), cul, t["state"], t["dy"],
                       t["dl"], True, zoh) for t in (w, m))
    for n in ("dx", "dB", "dC"):
        within(got[n], BF * ref[n].abs() + REST * mag[n] + TINY, ref[n], n)
    near(got["ddt"], ref["ddt"], BF + 2.0 ** -14, "ddt")
    for n in ("dA", "ddt_bias", "dDskip"):
        near(got[n], ref[n], 2.0 ** -14, n)
    within(got["dstate"], 2.0 ** -15 * mag["dstate"] + TINY, ref["dstate"], "dstate")


@pytest.mark.parametrize("N,H,lens", [(128, 24, [5, 1, 17] * 30 + [2000, 64]), (64, 20, [3] * 100 + [700, 1, 600]),
                                      (256, 24, [2] * 50 + [900])])
def test_segments_among_many_sequences(N, H, lens):
    torch, c, cu, cul, w, m = scan_inputs(80 + N, lens, H, 1, N)
    cps, blocks, full = scan_plan(cul[-1], len(lens), H, 1, N)
    check_workspaces(cul[-1], len(lens), H, 1, N)
    assert full and max(lens) > 2 * cps * 64, (cps, blocks)          # the longest has three segments or more
    out = torch.empty_like(c["state"])
    y = ssm().ssd_packed_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], cu, c["bias"], c["D"], state=c["state"], state_out=out)
    got = ssm().ssd_packed_bwd(c["x"], c["dt"], c["A"], c["B"], c["C"], c["dy"], cu, c["bias"], c["D"], state=c["state"],
                               dstate_out=c["dl"])
    torch.cuda.synchronize()
    names = ("x", "dt", "A", "B", "C", "bias", "D")
    ref, last, mag = on_gpu(R.ssd, *(w[k] for k in names), cul, w["state"])
    big = on_gpu(R.ssd, *(m[k] for k in names), cul, m["state"])[1]
    within(y, BF * ref.abs() + REST * mag + TINY, ref, "y")
    within(out, 2.0 ** -15 * big + TINY, last, "state")
    gr, gm = (on_gpu(R.ssd_grads, *(t[k] for k in names), cul, t["state"], t["dy"], t["dl"]) for t in (w, m))
    for n in ("dx", "dB", "dC"):
        within(got[n], BF * gr[n].abs() + REST * gm[n] + TINY, gr[n], n)
    within(got["dstate"], 2.0 ** -15 * gm["dstate"] + TINY, gr["dstate"], "dstate")
    for n in ("dA", "ddt_bias", "dDskip"):
        near(got[n], gr[n], 2.0 ** -14, n)


def conv_tiles(tokens, dim, width, elem):
    """Tokens per tile of the forward and of the backward, for 16-byte aligned rows."""
    v = 16 // elem
    lanes = up(dim, v)
    fwd = min(max(tokens * lanes // (2 * 1024 * 64), 8), 64) // 8 * 8
    across = up(dim, v * 64)
    cost = {t: up(up(tokens, t) * across, 1024) * (t + width - 1 + 8) for t in range(8, 72, 8)}
    return fwd, min(cost, key=lambda t: (cost[t], t))


@pytest.mark.parametrize("dtype,D,width,lens", [
    ("bf16", 4104, 4, [4000, 1, 0, 2, 6123, 3, 2871]), ("bf16", 5376, 4, [1, 8000, 40, 150, 8300]),
    ("bf16", 5376, 3, [1200, 3, 5000, 1, 1987]), ("f32", 2052, 2, [9000, 0, 7, 6900]),
])
def test_long_tiles_of_the_convolution(dtype, D, width, lens):
    torch = T()
    r = Rand(90 + D + width)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cu, cul, rows = packed(lens)
    fwd, bwd = conv_tiles(rows, D, width, dt.itemsize)
    assert fwd >= 32 and bwd >= 32 and (rows % fwd or rows % bwd), (fwd, bwd)
    x, du = r(rows, D, dtype=dt), r(rows, D, dtype=dt)
    w, b, state = r(D, width, scale=0.5), r(D, scale=0.2), r(len(lens), D, width - 1)
    out = torch.empty_like(state)
    u = ssm().conv1d_packed_fwd(x, w, cu, b, state=state, state_out=out)
    got = ssm().conv1d_packed_bwd(x, w, du, cu, b, state=state, want_dstate=True)
    torch.cuda.synchronize()
    # the definition, a sequence at a time
    ref = {k: torch.empty(rows, D, dtype=torch.float64, device="cuda") for k in ("u", "mag", "dx")}
    dw, db, first = torch.zeros_like(w).double(), torch.zeros_like(b).double(), torch.empty_like(state).double()
    wd, bd = w.double(), b.double()
    for s, (a, e) in enumerate(zip(cul, cul[1:])):
        n = e - a
        row = torch.cat([state[s].double().T, x[a:e].double()])
        taps = [row[k:k + n] * wd[:, k] for k in range(width)]
        pre = sum(taps) + bd
        ref["mag"][a:e] = sum(t.abs() for t in taps) + bd.abs()
        ref["u"][a:e] = R.silu(pre)
        dpre = du[a:e].double() * R.silu_slope(pre)
        drow = torch.zeros_like(row)
        for k in range(width):
            drow[k:k + n] += dpre * wd[:, k]
            dw[:, k] += (dpre * row[k:k + n]).sum(0)
        db += dpre.sum(0)
        ref["dx"][a:e], first[s] = drow[width - 1:], drow[:width - 1].T
        assert torch.equal(out[s], row[n:].T.float())
    half = BF if dt.itemsize == 2 else HALF32
    ref = {k: v.cpu() for k, v in ref.items()}
    within(u, half * ref["u"].abs() + 2.0 ** -20 * ref["mag"] + 1e-30, ref["u"], "u")
    near(got["dx"], ref["dx"], (BF if dt.itemsize == 2 else 0) + 2.0 ** -19, "dx")
    # sums of thousands of terms of either sign: fp32 runs of at most 64 and of the tiles, 2^-24 sqrt(n) of the terms' norm
    for n, v in (("dweight", dw), ("dbias", db), ("dstate", first)):
        near(got[n], v.cpu(), 2.0 ** -18, n)


@pytest.mark.parametrize("dtype,rows,n,groups,gate,center", [
    ("bf16", 4500, 5120, 1, "first", False), ("bf16", 1100, 4096, 2, "behind", True), ("bf16", 1300, 16384, 1, "first", True),
    ("bf16", 300, 16384, 1, "behind", False), ("f32", 1100, 5120, 1, "first", True), ("f32", 300, 16384, 1, None, False),
    ("bf16", 700, 5001, 1, "first", False), ("bf16", 5000, 1024, 2, "first", False),
])
def test_norm_over_several_rows(dtype, rows, n, groups, gate, center):
    torch = T()
    r = Rand(100 + n + rows)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    D = n * groups
    v = (16 // dt.itemsize) if n % (16 // dt.itemsize) == 0 else 1
    team = next(t for t, k in ((64, 4), (256, 16 if v == 1 else 32 // v), (1024, 32)) if v * t * k >= n)
    assert rows > up(2048 // max(team // 64, 4), groups) * (4 if team == 64 else 1)     # the backward's workgroups take several rows
    x, dy = r(rows, D, dtype=dt), r(rows, D, dtype=dt)
    z = r(rows, D, dtype=dt) if gate else None
    w, b = 1 + r(D, scale=0.2), r(D, scale=0.3)
    y = ssm().gated_norm_fwd(x, w, b, z, groups=groups, gate_first=gate == "first", center=center)
    got = ssm().gated_norm_bwd(x, w, dy, b, z, groups=groups, gate_first=gate == "first", center=center)
    torch.cuda.synchronize()
    wide = [None if t is None else t.double() for t in (x, w, b, z)]
    ref = R.norm(*wide, groups, 1e-5, gate == "first", center).cpu()
    tol = (BF if dt.itemsize == 2 else 0) + 2.0 ** -18
    within(y, tol * (ref.abs() + w.cpu().double().abs() + b.cpu().double().abs()), ref, "y")
    near(y, ref, tol, "y")
    g = R.norm_grads(*wide, groups, 1e-5, gate == "first", center, dy.double())
    for name in ("dx", "dz"):
        if g[name] is not None:
            near(got[name], g[name].cpu(), (BF if dt.itemsize == 2 else 0) + 2.0 ** -17, name)
    near(got["dweight"], g["dweight"].cpu(), 2.0 ** -17, "dweight")
    near(got["dbias"], g["dbias"].cpu(), 2.0 ** -17, "dbias")
