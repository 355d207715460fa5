"""The packed Mamba-2 block operators as they are used: one behind the other, in prompts, single tokens and gradients;
captured into graphs; on other streams; with NaN in what a call must not use; with offsets past 32 bits; and the calls
that the Python forms refuse.

Tolerances: test_packed_gpu.py's, a rounding of a stage's output (2^-8 in bf16) counted once for every factor that
carries it on.
"""
import ctypes

import pytest

import packed_ref as R
from test_packed_gpu import BF, TOL_STATE, Rand, T, f64, last_pool, near, packed, ssm

pytestmark = pytest.mark.gpu


class Block:
    """Parameters of one block, and its run: a projection's rows hold [z, x B C, dt]."""

    def __init__(self, r, H, G, N, groups):
        import torch
        self.H, self.G, self.N, self.groups = H, G, N, groups
        self.I, self.D = H * 64, H * 64 + 2 * G * N
        self.width = self.I + self.D + 8 * ((H + 7) // 8)
        self.w, self.b = r(self.D, 4, scale=0.5), r(self.D, scale=0.2)
        self.A = -torch.exp(torch.rand(H, generator=r.g) * 2.0).cuda()
        self.bias, self.skip = (torch.rand(H, generator=r.g) * 3 - 4).cuda(), 1 + r(H, scale=0.1)
        self.g = 1 + r(self.I, scale=0.2)

    def cut(self, rows):
        return rows[:, :self.I], rows[:, self.I:self.I + self.D], rows[:, self.I + self.D:self.I + self.D + self.H]

    def heads(self, u):
        i, gn = self.I, self.G * self.N
        return (u[:, :i].unflatten(1, (self.H, 64)), u[:, i:i + gn].unflatten(1, (self.G, self.N)),
                u[:, i + gn:].unflatten(1, (self.G, self.N)))

    def prompt(self, rows, cu, conv, state, idx, has, **kw):
        z, xbc, dt = self.cut(rows)
        u = ssm().conv1d_packed_fwd(xbc, self.w, cu, self.b, state=conv, state_out=conv, state_idx=idx, has_state=has, **kw)
        x, B, C = self.heads(u)
        y = ssm().ssd_packed_fwd(x, dt, self.A, B, C, cu, self.bias, self.skip, state=state, state_out=state,
                                 state_idx=idx, has_state=has, **kw)
        return u, y, ssm().gated_norm_fwd(y.flatten(1), self.g, z=z, groups=self.groups, **kw)

    def tokens(self, rows, conv, state, idx, **kw):
        z, xbc, dt = self.cut(rows)
        x, B, C = self.heads(ssm().conv1d_slot_update(conv, xbc, self.w, self.b, state_idx=idx, **kw))
        y = ssm().ssd_slot_update(state, x, dt, self.A, B, C, self.bias, self.skip, state_idx=idx, **kw)
        return ssm().gated_norm_fwd(y.flatten(1), self.g, z=z, groups=self.groups, **kw)

    def grads(self, rows, cu, u, y, dout, conv, state, idx, has, **kw):
        """Gradients of the rows (side by side, as the projection's backward takes them), of states and parameters."""
        import torch
        z, xbc, dt = self.cut(rows)
        drows = torch.zeros_like(rows)
        dz, dxbc, ddt = self.cut(drows)
        n = ssm().gated_norm_bwd(y.flatten(1), self.g, dout, z=z, groups=self.groups, dz=dz, **kw)
        du = torch.zeros_like(u)
        dx, dB, dC = self.heads(du)
        x, B, C = self.heads(u)
        s = ssm().ssd_packed_bwd(x, dt, self.A, B, C, n["dx"].view(-1, self.H, 64), cu, self.bias, self.skip, state=state,
                                 state_idx=idx, has_state=has, out=dict(dx=dx, dB=dB, dC=dC, ddt=ddt), **kw)
        c = ssm().conv1d_packed_bwd(xbc, self.w, du, cu, self.b, state=conv, state_idx=idx, has_state=has,
                                    want_dstate=True, dx=dxbc, **kw)
        return dict(drows=drows, dg=n["dweight"], dA=s["dA"], dbias=s["ddt_bias"], dskip=s["dDskip"], dstate=s["dstate"],
                    dw=c["dweight"], db=c["dbias"], dconv=c["dstate"])

    # in 64 bits
    def ref(self, rows, cu, conv, state):
        z, xbc, dt = self.cut(f64(rows))
        _, u, lastw = R.conv(xbc, f64(self.w), f64(self.b), cu, conv)
        x, B, C = self.heads(u)
        y, last, _ = R.ssd(x, dt, f64(self.A), B, C, f64(self.bias), f64(self.skip), cu, state)
        return u, y, R.norm(y.flatten(1), f64(self.g), None, z, self.groups, 1e-5, True, False), lastw, last

    def ref_grads(self, rows, cu, conv, state, dout):
        z, xbc, dt = self.cut(f64(rows))
        u, y, _, _, _ = self.ref(rows, cu, conv, state)
        x, B, C = self.heads(u)
        n = R.norm_grads(y.flatten(1), f64(self.g), None, z, self.groups, 1e-5, True, False, f64(dout))
        s = R.ssd_grads(x, dt, f64(self.A), B, C, f64(self.bias), f64(self.skip), cu, state,
                        n["dx"].view(-1, self.H, 64), None)
        import torch
        c = R.conv_grads(xbc, f64(self.w), f64(self.b), cu, conv, torch.cat([s[k].flatten(1) for k in ("dx", "dB", "dC")], 1),
                         None)
        return dict(drows=torch.cat([n["dz"], c["dx"], s["ddt"]], 1), dg=n["dweight"], dA=s["dA"], dbias=s["ddt_bias"],
                    dskip=s["dDskip"], dstate=s["dstate"], dw=c["dweight"], db=c["dbias"], dconv=c["dstate"])


def setup(seed, lens, H=6, G=2, N=64, groups=3, slots=None):
    torch = T()
    r = Rand(seed)
    k = Block(r, H, G, N, groups)
    cu, cul, rows = packed(lens)
    S = len(lens)
    x = r(rows, k.width, dtype=torch.bfloat16)
    slots = slots or S + 2
    idx = torch.randperm(slots, generator=r.g)[:S].to(torch.int32).cuda()
    return torch, r, k, cu, cul, x, idx, r(slots, k.D, 3), r(slots, H, 64, N)


def test_prompt_then_tokens():
    """Prompts, some of them continued, and the tokens behind them one at a time: the same outputs and states as over the
    whole sequences at once in 64 bits."""
    torch, r, k, cu, cul, x, idx, conv, state = setup(1, [70, 9, 1, 130])
    S, more = 4, 5
    has = torch.tensor([True, False, False, True]).cuda()
    first_c = R.first_states(S, (k.D, 3), conv, idx, has)
    first_s = R.first_states(S, (k.H, 64, k.N), state, idx, has)
    ahead = [r(S, k.width, dtype=torch.bfloat16) for _ in range(more)]
    _, _, out = k.prompt(x, cu, conv, state, idx, has)
    outs = [k.tokens(a, conv, state, idx) for a in ahead]
    torch.cuda.synchronize()
    # whole sequences: each prompt and its tokens
    rows, where = [], []
    for s in range(S):
        where.append((sum(len(a) for a in rows), cul[s + 1] - cul[s]))
        rows += [x[cul[s]:cul[s + 1]]] + [a[s:s + 1] for a in ahead]
    total = [0]
    for s in range(S):
        total.append(total[-1] + where[s][1] + more)
    _, _, ref, lastw, last = k.ref(torch.cat(rows), total, first_c, first_s)
    got = []
    for s in range(S):
        got += [out[cul[s]:cul[s + 1]]] + [o[s:s + 1] for o in outs]
    # x, B and C are rounded (three factors of every term), then three roundings of the scan, the norm's one
    near(torch.cat(got), ref, 7 * BF, "out")
    # two rounded factors, x and B, and the scan's own
    near(state[idx.long()], last, 2 * BF + TOL_STATE, "state")
    assert torch.equal(f64(conv[idx.long()]), lastw)


@pytest.mark.parametrize("H,G,N,groups", [(6, 2, 64, 3), (4, 1, 128, 1)])
def test_gradients_of_the_block(H, G, N, groups):
    torch, r, k, cu, cul, x, idx, conv, state = setup(2, [65, 1, 40, 0, 129], H, G, N, groups)
    has = torch.tensor([True, False, True, False, True]).cuda()
    first_c = R.first_states(5, (k.D, 3), conv, idx, has)
    first_s = R.first_states(5, (k.H, 64, k.N), state, idx, has)
    keep = conv.clone(), state.clone()
    u, y, out = k.prompt(x, cu, conv, state, idx, has)
    dout = r(x.shape[0], k.I, dtype=torch.bfloat16)
    got = k.grads(x, cu, u, y, dout, *keep, idx, has)
    torch.cuda.synchronize()
    ref = k.ref_grads(x, cul, first_c, first_s, dout)
    got["drows"] = got["drows"][:, :ref["drows"].shape[1]]
    # y (6 roundings in front of the norm's gradients) and dy = the norm's dx (one more, and its y, z: 7 + 1) are the inputs
    # of the scan's, with x, B, C (3) and the scan's own 3, then du's, dx's: 16 at most, in bf16
    for n in ref:
        near(got[n], ref[n], 16 * BF, n)


def test_captured_block():
    """Prompt, tokens and gradients captured into one graph and replayed on changed inputs, lengths, slots and states, with
    eager work between: every replay is the eager result, bit for bit."""
    torch, r, k, cu, cul, x, idx, conv, state = setup(3, [100, 28, 72], N=128)
    has = torch.tensor([True, True, False]).cuda()
    tok, dout = r(3, k.width, dtype=torch.bfloat16), r(200, k.I, dtype=torch.bfloat16)

    def work(conv, state):
        c0, s0 = conv.clone(), state.clone()
        u, y, out = k.prompt(x, cu, conv, state, idx, has)
        g = k.grads(x, cu, u, y, dout, c0, s0, idx, has)
        return dict(g, out=out, tokens=k.tokens(tok, conv, state, idx), conv=conv, state=state)

    work(conv.clone(), state.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fixed = conv.clone(), state.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        outs = work(*fixed)
    for lens, slots, on in (([100, 28, 72], None, [1, 1, 0]), ([1, 198, 1], [4, 0, 2], [0, 1, 1]),
                            ([0, 64, 100], [1, 4, 3], [1, 0, 1]), ([200, 0, 0], [2, 1, 0], [0, 0, 0])):
        x.copy_(r(200, k.width, dtype=torch.bfloat16))
        dout.copy_(r(200, k.I, dtype=torch.bfloat16))
        cu.copy_(packed(lens)[0])
        n = sum(lens)
        x[n:] = 0
        if slots:
            idx.copy_(torch.tensor(slots, dtype=torch.int32))
        has.copy_(torch.tensor(on, dtype=torch.bool))
        c, s = r(*conv.shape), r(*state.shape)
        fixed[0].copy_(c)
        fixed[1].copy_(s)
        want = work(c, s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for m in want:
            if m == "dg" and n < 200:    # (the norm takes every row, also those that the scan leaves unset)
                continue
            a, b = outs[m], want[m]
            a, b = (a[:n], b[:n]) if a.shape[0] == 200 else (a, b)
            assert torch.equal(a, b), (lens, m)


def test_other_stream_and_two_at_once():
    """Calls on two streams at once, by ``stream`` and by the current stream, are the calls one behind the other."""
    torch, r, k, cu, cul, x, idx, conv, state = setup(4, [300, 5, 207], N=128)
    x2, dout = r(*x.shape, dtype=torch.bfloat16), r(512, k.I, dtype=torch.bfloat16)

    def work(rows, **kw):
        c, s = conv.clone(), state.clone()
        u, y, out = k.prompt(rows, cu, c, s, idx, None, **kw)
        return [out, c, s] + list(k.grads(rows, cu, u, y, dout, conv, state, idx, None, **kw).values())

    want = work(x), work(x2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            one = work(x)
        with torch.cuda.stream(b):
            two = work(x2)
        torch.cuda.synchronize()
        for got, ref in zip((one, two), want):
            assert all(torch.equal(p, q) for p, q in zip(got, ref))
    # by argument: the caller orders the streams
    b.wait_stream(torch.cuda.current_stream())
    out = ssm().gated_norm_fwd(dout, k.g, stream=b)
    u = ssm().conv1d_packed_fwd(k.cut(x)[1], k.w, cu, k.b, stream=b)
    torch.cuda.current_stream().wait_stream(b)
    assert torch.equal(out, ssm().gated_norm_fwd(dout, k.g)) and torch.equal(u, ssm().conv1d_packed_fwd(k.cut(x)[1], k.w, cu, k.b))


def test_what_is_not_used_may_be_nan():
    """NaN in rows outside the sequences, in a neighbouring sequence, in slots that are not named or not started from, and
    in rows behind the last one of a tile reaches nothing else."""
    torch, r, k, cu, cul, x, idx, conv, state = setup(5, [70, 50, 33, 0, 129], N=128)
    S = 5
    cu2, cul2, rows2 = packed([70, 50, 33, 0, 129], lead=3, tail=9)
    has = torch.tensor([True, True, False, True, True]).cuda()
    dout = r(x.shape[0], k.I, dtype=torch.bfloat16)
    nan = float("nan")

    def work(poison):
        c, s = conv.clone(), state.clone()
        rows = torch.zeros(rows2, k.width, dtype=torch.bfloat16, device="cuda")
        rows[3:-9] = x
        d = torch.zeros(rows2, k.I, dtype=torch.bfloat16, device="cuda")
        d[3:-9] = dout
        if poison:
            named = set(idx.tolist())
            for t in (c, s):
                for n in range(t.shape[0]):
                    if n not in named:
                        t[n] = nan
                t[int(idx[2])] = nan               # has_state False
            for t in (rows, d):
                t[:3], t[-9:] = nan, nan
        if poison == "neighbour":
            rows[cul2[1]:cul2[2]] = nan
        c0, s0 = c.clone(), s.clone()
        u, y, out = k.prompt(rows, cu2, c, s, idx, has)
        return u, y, out, c, s, k.grads(rows, cu2, u, y, d, c0, s0, idx, has)

    clean = work(None)
    for how in ("outside", "neighbour"):
        got = work(how)
        torch.cuda.synchronize()
        for s in range(S):
            if how == "neighbour" and s == 1:
                assert bool(got[0][cul2[1]:cul2[2]].isnan().all())
                continue
            a, e = cul2[s], cul2[s + 1]
            for g, w in zip(got[:3], clean[:3]):
                assert torch.equal(g[a:e], w[a:e]), (how, s)
            n = int(idx[s])
            assert torch.equal(got[3][n], clean[3][n]) and torch.equal(got[4][n], clean[4][n])
            assert torch.equal(got[5]["drows"][a:e], clean[5]["drows"][a:e]), (how, s)
            assert torch.equal(got[5]["dstate"][s], clean[5]["dstate"][s])
            assert torch.equal(got[5]["dconv"][s], clean[5]["dconv"][s])
        if how == "outside":
            # (the norm takes every row, so its weight gradient is not the sequences' alone)
            for n in ("dA", "dbias", "dskip", "dw", "db"):
                assert torch.equal(got[5][n], clean[5][n]), n


def test_extreme_steps_stay_finite():
    """Steps that decay everything or nothing, next to each other in a chunk."""
    torch, r, k, cu, cul, x, idx, conv, state = setup(6, [130, 64], N=64)
    z, xbc, dt = k.cut(x)
    dt[:] = torch.tensor([1e4, -1e4, 0.0, 50.0, -60.0])[torch.randint(0, 5, dt.shape, generator=r.g)].to(dt.dtype).cuda()
    dt[64:70] = 1e4
    u, y, out = k.prompt(x, cu, conv, state, idx, None)
    g = k.grads(x, cu, u, y, r(194, k.I, dtype=torch.bfloat16), conv, state, idx, None)
    for t in (y, out, state, *g.values()):
        assert bool(t.isfinite().all())


def test_offsets_past_32_bits():
    """Rows more than 2^31 bytes into their tensors and slots more than 2^32 into the pool."""
    torch = T()
    r = Rand(7)
    H, G, N, n = 2, 1, 64, 600
    far = torch.empty(n, 1 << 22, dtype=torch.bfloat16, device="cuda")            # 5 GB
    D = H * 64 + 2 * G * N
    near_ = r(n, D + 8, dtype=torch.bfloat16)
    far[:, :D + 8] = near_
    cu, cul, _ = packed([299, 301])
    w, b, A = r(D, 4), r(D), -torch.rand(H, generator=r.g).cuda() - 0.1
    slots = 140000
    big = torch.empty(slots, H, 64, N, device="cuda")                              # 4.6 GB
    idx = torch.tensor([slots - 1, 3], dtype=torch.int32).cuda()
    start = r(2, H, 64, N)
    big[idx.long()] = start
    small = start.clone()

    def cut(t):
        return (t[:, :H * 64].unflatten(1, (H, 64)), t[:, D:D + H], A, t[:, H * 64:H * 64 + N].unflatten(1, (1, N)),
                t[:, H * 64 + N:D].unflatten(1, (1, N)))

    got = ssm().conv1d_packed_fwd(far[:, :D], w, cu, b)
    assert torch.equal(got, ssm().conv1d_packed_fwd(near_[:, :D], w, cu, b))
    dg, dn = (ssm().conv1d_packed_bwd(t[:, :D], w, t[:, 8:D + 8], cu, b) for t in (far, near_))
    assert all(torch.equal(dg[m], dn[m]) for m in ("dx", "dweight", "dbias"))
    x2, nx = (ssm().gated_norm_fwd(t[:, :D], b, z=t[:, 8:D + 8]) for t in (far, near_))
    assert torch.equal(x2, nx)
    dy = r(n, H, 64, dtype=torch.bfloat16)
    ga, gb = (ssm().ssd_packed_bwd(*cut(t), dy, cu, state=p, state_idx=i) for t, p, i in ((far, big, idx), (near_, small, None)))
    assert all(torch.equal(ga[m], gb[m]) for m in ("dx", "ddt", "dA", "dB", "dC", "dstate"))
    ya = ssm().ssd_packed_fwd(*cut(far), cu, state=big, state_out=big, state_idx=idx)
    yb = ssm().ssd_packed_fwd(*cut(near_), cu, state=small, state_out=small)
    assert torch.equal(ya, yb) and torch.equal(big[idx.long()], small)
    sa = ssm().ssd_slot_update(big, *(t if t is A else t[:2] for t in cut(far)), state_idx=idx)
    sb = ssm().ssd_slot_update(small, *(t if t is A else t[:2] for t in cut(near_)))
    assert torch.equal(sa, sb) and torch.equal(big[idx.long()], small)


@pytest.mark.parametrize("lens", [[200, 3, 0, 65, 1, 64, 128, 129] * 4, [63, 65] * 9 + [700], [66] * 40, [1, 640, 1]])
def test_cut_sequences_among_short_ones(lens):
    """Segments of one chunk, kept states side by side, against no segments at all; nothing behind the workspace is
    written."""
    torch, r, k, cu, cul, x, idx, conv, state = setup(9, lens, H=3, G=1, groups=1)
    S = len(lens)
    dy, dl = r(x.shape[0], 3, 64, dtype=torch.bfloat16), r(S, 3, 64, 64, scale=0.3)
    z, xbc, dt = k.cut(x)
    xs, B, C = k.heads(xbc)
    args = (xs, dt, k.A, B, C)
    m = ssm()

    def run(chunks, fwd, bwd):
        out = state.clone()
        y = m.ssd_packed_fwd(*args, cu, k.bias, k.skip, state=state, state_out=out, state_idx=idx, segment_chunks=chunks,
                             workspace=fwd)
        return dict(m.ssd_packed_bwd(*args, dy, cu, k.bias, k.skip, state=state, state_idx=idx, dstate_out=dl,
                                     segment_chunks=chunks, workspace=bwd), y=y, state=out)

    def space(name, chunks):
        p = m._abi.SsdPackedParams(ntokens=x.shape[0], nseqs=S, nheads=3, headdim=64, ngroups=1, dstate=64, nslots=S + 2,
                                   io_dtype=m.SSM_BF16, dt_softplus=1, segment_chunks=chunks)
        n = int(getattr(m._abi.lib(), name)(ctypes.byref(p)))
        return torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda"), n

    wf, nf = space("ssm_ssd_packed_fwd_workspace_bytes", 1)
    wb, nb = space("ssm_ssd_packed_bwd_workspace_bytes", 1)
    got, ref = run(1, wf, wb), run(1000, None, None)
    torch.cuda.synchronize()
    assert bool((wf[nf:] == 7).all()) and bool((wb[nb:] == 7).all())
    # each side is within its own tolerance of the same 64-bit values
    for n, tol in (("y", 3 * BF), ("dx", 3 * BF), ("dB", 3 * BF), ("dC", 3 * BF), ("ddt", BF + 2.0 ** -14),
                   ("state", TOL_STATE), ("dstate", TOL_STATE), ("dA", 2.0 ** -14), ("ddt_bias", 2.0 ** -14)):
        near(got[n], f64(ref[n]), 2 * tol, n)


def test_refusals():
    torch = T()
    r = Rand(8)
    m, bf = ssm(), torch.bfloat16
    x, w, cu = r(10, 16, dtype=bf), r(16, 4), packed([4, 6])[0]
    H, N = 2, 64
    h, g, dt, A = r(10, H, 64, dtype=bf), r(10, 1, N, dtype=bf), r(10, H, dtype=bf), -torch.ones(H).cuda()
    conv, state = r(2, 16, 3), r(2, H, 64, N)
    ok = dict(x=x, conv_w=w, cu_seqlens=cu)
    for kw in (dict(x=x.half()), dict(x=x.t()), dict(conv_w=w.cpu()), dict(conv_w=w[:8]), dict(conv_w=w.to(bf)),
               dict(conv_w=r(16, 5)), dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:1]), dict(cu_seqlens=cu.cpu()),
               dict(conv_bias=r(8)), dict(state=conv[:1]), dict(state=conv, state_out=r(3, 16, 3)),
               dict(state=conv.to(bf)), dict(state=r(2, 16, 4)), dict(state=conv, state_idx=cu[:2].long()),
               dict(state=conv, state_idx=cu), dict(state=conv, has_state=cu[:2]), dict(u=x), dict(u=x[:5]),
               dict(u=x.float()), dict(state=r(3, 16, 3)[:2], state_out=conv, u=r(10, 8, dtype=bf))):
        with pytest.raises((ValueError, TypeError, m.SSMError)):
            m.conv1d_packed_fwd(**{**ok, **kw})
    wide = r(10, 24, dtype=bf)
    with pytest.raises(ValueError, match="overlap"):
        m.conv1d_packed_fwd(wide[:, :16], w, cu, u=wide[:, 8:])
    with pytest.raises(ValueError, match="overlap"):
        pool = r(5, 16, 3)
        m.conv1d_packed_fwd(x, w, cu, state=pool[:4], state_out=pool[1:])
    with pytest.raises(ValueError):
        m.conv1d_slot_update(None, x, w)
    with pytest.raises(ValueError):
        m.conv1d_slot_update(conv, x, w)                               # ten rows, two slots
    with pytest.raises((ValueError, m.SSMError)):
        m.conv1d_packed_bwd(x, w, x, cu, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(m.SSMError):
        m.conv1d_packed_bwd(x, w, x, cu, workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
    ok = dict(x=h, dt=dt, A=A, B=g, C=g, cu_seqlens=cu)
    odd = torch.empty(10 * 128 + 4, dtype=bf, device="cuda")[4:].view(10, H, 64)
    for kw in (dict(x=h.float()), dict(x=h[:, :, :32]), dict(dt=dt[:5]), dict(A=A.to(bf)), dict(B=g[:, 0]), dict(B=None),
               dict(C=r(10, 1, 128, dtype=bf)), dict(B=r(10, 1, 32, dtype=bf), C=r(10, 1, 32, dtype=bf)),
               dict(B=r(10, 3, 64, dtype=bf), C=r(10, 3, 64, dtype=bf)), dict(x=odd), dict(x=h.transpose(1, 2)),
               dict(Dskip=r(3)), dict(dt_bias=A.cpu()), dict(state=state[:1]), dict(state=r(2, H, 64, 128)),
               dict(disc=5), dict(segment_chunks=-1), dict(y=h), dict(x=h[:0], dt=dt[:0], B=g[:0], C=g[:0])):
        with pytest.raises((ValueError, TypeError, m.SSMError)):
            m.ssd_packed_fwd(**{**ok, **kw})
    for kw in (dict(dy=h[:5]), dict(dy=h.float()), dict(out=dict(dA=A)), dict(out=dict(dx=h)), dict(dstate_out=state[:1])):
        with pytest.raises((ValueError, TypeError, m.SSMError)):
            m.ssd_packed_bwd(**{**ok, "dy": r(10, H, 64, dtype=bf), **kw})
    both = r(10, 128, dtype=bf)
    with pytest.raises(ValueError, match="overlap"):
        m.ssd_packed_bwd(**ok, dy=h.clone(), out=dict(dB=both[:, :64].unflatten(1, (1, 64)),
                                                      dC=both[:, 32:96].unflatten(1, (1, 64))))
    for kw in (dict(weight=r(8)), dict(groups=3), dict(groups=0), dict(z=x[:5]), dict(eps=-1.0), dict(y=x[:, :8])):
        with pytest.raises((ValueError, TypeError, m.SSMError)):
            m.gated_norm_fwd(**{**dict(x=x, weight=r(16)), **kw})
    with pytest.raises(ValueError):
        m.gated_norm_bwd(x, r(16), x, dz=x.clone())
