"""The operators at a block's ends as they are used: around the packed Mamba-2 operators, in a projection's training step,
captured into graphs, on other streams, side by side; offsets past 32 bits; and the calls that the Python forms refuse.
"""
import pytest
import torch

import projection_ref as R
from test_projection_gpu import BF, F32, F8, Rand, inside, ssm, tolerance, u
from test_packed_use_gpu import Block

pytestmark = pytest.mark.gpu


class Ends:
    """A Mamba-2 block with its ends: norm with 8-bit output, input projection, the packed operators, output projection."""

    def __init__(self, r, D, H=4, G=1, N=64):
        from test_packed_gpu import Rand as PackedRand
        self.block = Block(PackedRand(11), H, G, N, 1)
        self.D, self.width = D, self.block.width
        self.w_norm = 1 + r(D, scale=0.1)
        self.w_in, self.w_out = r(self.width, D, scale=D ** -0.5), r(D, self.block.I, scale=self.block.I ** -0.5)
        self.q_in, self.q_out = ssm().quantize_fp8_blocks(self.w_in), ssm().quantize_fp8_blocks(self.w_out)

    def prompt(self, x, res, cu, conv, state, idx, has, **kw):
        q, h, s = ssm().add_norm_fwd(x, self.w_norm, res, y_dtype=F8, **kw)
        rows = ssm().matmul_fp8(q, s, self.q_in["q"], self.q_in["scale"], **kw)
        _, _, y = self.block.prompt(rows, cu, conv, state, idx, has, **kw)
        yq = ssm().quantize_fp8(y, **kw)
        return h, rows, y, ssm().matmul_fp8(yq["q"], yq["scale"], self.q_out["q"], self.q_out["scale"], **kw)

    def tokens(self, x, res, conv, state, idx, **kw):
        q, h, s = ssm().add_norm_fwd(x, self.w_norm, res, y_dtype=F8, **kw)
        rows = ssm().matmul_fp8(q, s, self.q_in["q"], self.q_in["scale"], **kw)
        y = self.block.tokens(rows, conv, state, idx, **kw)
        yq = ssm().quantize_fp8(y, **kw)
        return h, ssm().matmul_fp8(yq["q"], yq["scale"], self.q_out["q"], self.q_out["scale"], **kw)

    def pools(self, r, slots):
        b = self.block
        return r(slots, b.D, 3), r(slots, b.H, 64, b.N, scale=0.3)


def near_rel(got, want, tol):
    e = float((got.double() - want.double()).norm() / want.double().norm())
    assert e <= tol, e


def test_block_with_its_ends():
    """Prompts, then single tokens: each stage against 64 bits of what the stage before it handed on; the whole against the
    block with exact projections."""
    r = Rand(21)
    D, lens = 320, [70, 1, 0, 129, 33]
    T, S = sum(lens), len(lens)
    e = Ends(r, D)
    x, res = r(T, D, dtype=BF), r(T, D)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    conv, state = e.pools(r, S + 2)
    idx, has = torch.randperm(S + 2, device="cuda")[:S].int(), torch.tensor([True, False, True, False, True], device="cuda")
    conv2, state2 = conv.clone(), state.clone()
    h, rows, y, out = e.prompt(x, res, cu, conv, state, idx, has)
    hw, yw = R.add_norm(x, res, e.w_norm, 1e-5)
    inside(h, hw, 2 * u * hw.abs())
    q, _, s = ssm().add_norm_fwd(x, e.w_norm, res, y_dtype=F8)
    want, size = R.product(q, s, e.q_in["q"], e.q_in["scale"], 128)
    inside(rows, want, tolerance(q, s, e.q_in["q"], e.q_in["scale"], 128, BF, want, size))
    yq = ssm().quantize_fp8(y)
    want, size = R.product(yq["q"], yq["scale"], e.q_out["q"], e.q_out["scale"], 128)
    inside(out, want, tolerance(yq["q"], yq["scale"], e.q_out["q"], e.q_out["scale"], 128, BF, want, size))
    # exact projections: an e4m3 value is off by 2^-4 at most and by about 2^-5.2 on average, two of them in each product, and
    # the nonlinear operators between the projections pass on about what they get
    rows_w = (yw @ e.w_in.double().T).to(BF)
    near_rel(rows, rows_w, 2 * 2.0 ** -5)
    _, _, y_w = e.block.prompt(rows_w, cu, conv2, state2, idx, has)
    near_rel(out, y_w.double() @ e.w_out.double().T, 8 * 2.0 ** -5)
    xt, rt = r(S, D, dtype=BF), r(S, D)
    _, tok = e.tokens(xt, rt, conv, state, idx)
    rows_w = (R.add_norm(xt, rt, e.w_norm, 1e-5)[1] @ e.w_in.double().T).to(BF)
    near_rel(tok, e.block.tokens(rows_w, conv2, state2, idx).double() @ e.w_out.double().T, 8 * 2.0 ** -5)


@pytest.mark.parametrize("T,K,N", [(300, 256, 400), (1999, 768, 1100)])
def test_training_step_of_a_projection(T, K, N):
    """y = x W^T in 8 bits and its gradients, all from quantised operands: against 64 bits of the codes element by element, and
    against the exact gradients within the quantisation's errors."""
    r = Rand(T + K)
    x, W, dy = r(T, K, dtype=BF), r(N, K, scale=K ** -0.5), r(T, N, scale=1e-3, dtype=BF)
    xq = ssm().quantize_fp8(x, columns=True)
    wq = ssm().quantize_fp8_blocks(W, columns=True)
    gq = ssm().quantize_fp8(dy, columns=True)
    y = ssm().matmul_fp8(xq["q"], xq["scale"], wq["q"], wq["scale"])
    dx = ssm().matmul_fp8(gq["q"], gq["scale"], wq["qt"], wq["scale_t"])
    dW = ssm().matmul_fp8(gq["qt"], gq["scale_t"], xq["qt"], xq["scale_t"], out_dtype=F32)
    assert y.shape == (T, N) and dx.shape == (T, K) and dW.shape == (N, K)
    for got, a, sa, b, sb, rows, out in ((y, xq["q"], xq["scale"], wq["q"], wq["scale"], 128, BF),
                                        (dx, gq["q"], gq["scale"], wq["qt"], wq["scale_t"], 128, BF),
                                        (dW, gq["qt"], gq["scale_t"], xq["qt"], xq["scale_t"], 1, F32)):
        want, size = R.product(a, sa, b, sb, rows)
        inside(got, want, tolerance(a, sa, b, sb, rows, out, want, size))
    # two quantised factors of mean error 2^-5.2 each
    near_rel(y, x.double() @ W.double().T, 2 * 2.0 ** -5)
    near_rel(dx, dy.double() @ W.double(), 2 * 2.0 ** -5)
    near_rel(dW, dy.double().T @ x.double(), 2 * 2.0 ** -5)


def test_gradients_against_differences():
    """The loss of norm and projection along a direction: the gradients that the operators give and a difference quotient of
    the exact loss agree within the quantisation's errors."""
    r = Rand(31)
    T, D, N = 200, 384, 320
    x, res, w, W, c = r(T, D, dtype=BF), r(T, D), 1 + r(D, scale=0.1), r(N, D, scale=D ** -0.5), r(T, N, dtype=BF)
    y, h, _ = ssm().add_norm_fwd(x, w, res)
    wq, gq, yq = ssm().quantize_fp8_blocks(W, columns=True), ssm().quantize_fp8(c, columns=True), ssm().quantize_fp8(y, columns=True)
    dy = ssm().matmul_fp8(gq["q"], gq["scale"], wq["qt"], wq["scale_t"])
    dW = ssm().matmul_fp8(gq["qt"], gq["scale_t"], yq["qt"], yq["scale_t"], out_dtype=F32)
    g = ssm().add_norm_bwd(h, w, dy)

    def loss(e, of):
        v = {"x": x.double(), "w": w.double(), "W": W.double()}
        v[of] = v[of] + e * step[of]
        hh = v["x"] + res.double()
        n = hh * (hh.square().mean(1, keepdim=True) + 1e-5).rsqrt() * v["w"]
        return ((n @ v["W"].T) * c.double()).sum()
    # along the gradients themselves, so that nothing cancels: <g, g> against the slope of the loss
    step = {"x": g["dresidual"].double(), "w": g["dweight"].double(), "W": dW.double()}
    for of, v in step.items():
        e = 1e-5 / float(v.norm())
        slope = float((loss(e, of) - loss(-e, of)) / (2 * e))
        assert abs(slope / float(v.square().sum()) - 1) <= 2 * 2.0 ** -5, of


def test_captured():
    """A step of single tokens with its ends, captured once and replayed with other inputs, slots and eager work between."""
    r = Rand(41)
    D, S, slots = 256, 20, 24
    e = Ends(r, D)
    x, res, idx = r(S, D, dtype=BF), r(S, D), torch.arange(S, device="cuda").int()
    conv, state = e.pools(r, slots)
    big = r(700, D, dtype=BF)
    wq = e.q_in

    def step():
        h, out = e.tokens(x, res, conv, state, idx)
        g = ssm().add_norm_bwd(h, e.w_norm, out, res)
        q = ssm().quantize_fp8(big, columns=True)
        y = ssm().matmul_fp8(q["q"], q["scale"], wq["q"], wq["scale"])
        dw = ssm().matmul_fp8(q["qt"], q["scale_t"], q["qt"], q["scale_t"], out_dtype=F32)
        return [h, out, g["dx"], g["dresidual"], g["dweight"], y, dw]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        rr = Rand(50 + k)
        x.copy_(rr(S, D, dtype=BF))
        res.copy_(rr(S, D))
        big.copy_(rr(700, D, dtype=BF))
        idx.copy_(torch.randperm(slots, device="cuda")[:S].int())
        c0, s0 = e.pools(rr, slots)
        conv.copy_(c0)
        state.copy_(s0)
        want = [t.clone() for t in step()]
        wc, ws = conv.clone(), state.clone()
        conv.copy_(c0)
        state.copy_(s0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(conv, wc) and torch.equal(state, ws)


def test_other_streams():
    """Calls on a given stream, and two streams at once, give what the current stream gives, bit for bit, and again."""
    r = Rand(61)
    x, res, w, W = r(1500, 640, dtype=BF), r(1500, 640), 1 + r(640, scale=0.1), r(900, 640)
    wq = ssm().quantize_fp8_blocks(W)

    def work(stream=None):
        kw = {} if stream is None else {"stream": stream}
        q, h, s = ssm().add_norm_fwd(x, w, res, y_dtype=F8, **kw)
        y = ssm().matmul_fp8(q, s, wq["q"], wq["scale"], **kw)
        g = ssm().quantize_fp8(y, columns=True, **kw)
        dw = ssm().matmul_fp8(g["qt"], g["scale_t"], g["qt"], g["scale_t"], out_dtype=F32, **kw)
        b = ssm().add_norm_bwd(h, w, x, res, **kw)
        return [q.float(), h, s, y, dw, b["dx"], b["dresidual"], b["dweight"]] if stream is None else [q, h, s, y, dw, b["dx"], b["dresidual"], b["dweight"]]
    want = work()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [work(a), work(b), work(a), work(b)]
    torch.cuda.synchronize()
    for g in got:
        g[0] = g[0].float()
        for p, q in zip(g, want):
            assert torch.equal(p, q)


def test_offsets_past_32_bits():
    """Rows that begin more than 2^32 bytes behind the first one."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    r = Rand(71)
    apart = (1 << 23) - 16
    base = torch.zeros(700 * apart, dtype=torch.uint8, device="cuda").view(F8)
    a = base.view(700, apart)[:, :272]
    a.view(torch.uint8).copy_(r.codes(700, 272).view(torch.uint8))
    sa, b, sb = r.scales(700, 3), r.codes(300, 272), r.scales(3, 3)
    want = ssm().matmul_fp8(a.contiguous(), sa, b, sb)
    assert torch.equal(ssm().matmul_fp8(a, sa, b, sb), want)
    sbr = r.scales(700, 3)
    want = ssm().matmul_fp8(b, r.scales(300, 3).fill_(0.5), a.contiguous(), sbr, out_dtype=F32)
    assert torch.equal(ssm().matmul_fp8(b, r.scales(300, 3).fill_(0.5), a, sbr, out_dtype=F32), want)
    del base, a
    wide = torch.zeros(6 << 30, dtype=torch.uint8, device="cuda")
    x = wide.view(BF)[:3 * (1 << 30)].view(3, 1 << 30)[:, :500]
    x.copy_(r(3, 500))
    w, res = 1 + r(500, scale=0.1), r(3, 500)
    y, h, _ = ssm().add_norm_fwd(x, w, res)
    y2, h2, _ = ssm().add_norm_fwd(x.contiguous(), w, res)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    assert torch.equal(ssm().quantize_fp8(x)["q"].float(), ssm().quantize_fp8(x.contiguous())["q"].float())
    g = ssm().add_norm_bwd(h, w, x)
    g2 = ssm().add_norm_bwd(h, w, x.contiguous())
    assert torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dweight"], g2["dweight"])


def test_long_outputs():
    """A result of more than 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    r = Rand(72)
    M, N, K = 70001, 33000, 16
    a = torch.randint(-3, 4, (M, K), generator=r.g, device="cuda").float().to(F8)
    b = torch.randint(-3, 4, (N, K), generator=r.g, device="cuda").float().to(F8)
    out = ssm().matmul_fp8(a, torch.ones(M, 1, device="cuda"), b, torch.ones(-(-N // 128), 1, device="cuda"))
    for rows in (slice(0, 300), slice(35000, 35300), slice(M - 300, M)):
        assert torch.equal(out[rows], (a[rows].float() @ b.float().t()).to(BF))


def test_refusals():
    r = Rand(81)
    x, w, res = r(6, 256, dtype=BF), r(256), r(6, 256)
    q, s = r.codes(6, 256), r.scales(6, 2)
    b, sb = r.codes(300, 256), r.scales(3, 2)
    shape, kind = ValueError, TypeError
    n, g, qz, mm = ssm().add_norm_fwd, ssm().add_norm_bwd, ssm().quantize_fp8, ssm().matmul_fp8
    y8 = torch.empty(6, 256, device="cuda").to(F8)
    calls = [
        (shape, lambda: n(x, w[:255])), (shape, lambda: n(x, w, res[:5])), (kind, lambda: n(x.half(), w)), (kind, lambda: n(x, w.to(BF))),
        (kind, lambda: n(x, w, res.half())), (kind, lambda: n(x, w, y_dtype=F32)), (kind, lambda: n(x, w, y_dtype=torch.float8_e5m2)),
        (kind, lambda: n(x, w, res, residual_dtype=BF)), (kind, lambda: n(x, w, res, residual_out=torch.empty_like(x))),
        (kind, lambda: n(x, w, y=y8, y_dtype=BF)), (shape, lambda: n(x, w, y_scale=s)), (shape, lambda: n(x, w, y_dtype=F8, y_scale=s[:, :1])),
        (shape, lambda: n(x, w, res, y=torch.empty(6, 255, device="cuda", dtype=BF))), (shape, lambda: n(x.t(), r(6))),
        (shape, lambda: n(x, w, x, y=x, residual_out=x)),                        # two outputs in one place
        (shape, lambda: n(x, w, r(6, 512)[:, ::2])), (shape, lambda: n(x, None)),
        (shape, lambda: n(x.float(), w, res, y=res)),                            # y over the residual
        (shape, lambda: g(res, w, x[:5])), (shape, lambda: g(res, w, None)), (kind, lambda: g(res, w, x, x)), (shape, lambda: g(res, w[1:], x)),
        (kind, lambda: g(res, w, x, dx=res)), (shape, lambda: g(x, w, x, dx=x, dresidual=x)),
        (shape, lambda: g(res, w, x, dx=res.view(BF)[:, 1:257])),                # dx inside h
        (shape, lambda: qz(x, rows=False)), (shape, lambda: qz(x, qt=q)), (shape, lambda: qz(x, rows=False, columns=True, q=q)),
        (kind, lambda: qz(x, q=x)), (shape, lambda: qz(x, q=q[:5])), (kind, lambda: qz(x.half())), (shape, lambda: qz(x, scale=s[:, :1])),
        (shape, lambda: qz(x, scale=x.view(F32)[:, :2])),                        # scales over x
        (shape, lambda: mm(q, s, b[:, :240], sb)), (shape, lambda: mm(q, s[:5], b, sb)), (shape, lambda: mm(q, s, b, sb[:2])),
        (kind, lambda: mm(q.float(), s, b, sb)), (kind, lambda: mm(q, s.double(), b, sb)), (shape, lambda: mm(q, s, b, None)),
        (shape, lambda: mm(q, s, None, sb)), (shape, lambda: mm(q, None, b, sb)), (kind, lambda: mm(q, s, b, sb, out_dtype=torch.float16)),
        (kind, lambda: mm(q, s, b, sb, out=torch.empty(6, 300, device="cuda"), out_dtype=BF)),
        (shape, lambda: mm(q, s, b, sb, out=torch.empty(6, 299, device="cuda"))), (shape, lambda: mm(q, s, b.cpu(), sb)),
        (shape, lambda: mm(q, s, q, s, out=q.view(BF)[:, :6])),                  # the result over an operand
    ]
    for i, (error, f) in enumerate(calls):
        with pytest.raises(error):
            f()
        torch.cuda.synchronize()
    E = ssm().SSMError
    odd = torch.empty(6, 257, dtype=torch.uint8, device="cuda").view(F8)
    for f in (lambda: mm(odd[:, :256], s, b, sb),                                # rows off 16 bytes
              lambda: mm(q[:, :250], s, b[:, :250], sb),                         # k no multiple of 16
              lambda: n(r(2, 16385), r(16385)), lambda: n(x, w, eps=-1.0), lambda: n(x[:0], w), lambda: qz(x[:0]), lambda: qz(x[:, :0]),
              lambda: mm(q[:0], s[:0], b, sb), lambda: g(res, w, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
              lambda: qz(x, q=odd[:, :256])):
        with pytest.raises(E):
            f()


def test_more_rows_than_a_launch():
    """A row more than 2^23 workgroups of four rows: every one is quantised, the last like the first."""
    rows = (1 << 25) + 3
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    x = torch.arange(rows, device="cuda", dtype=torch.float32)[:, None].remainder(1000).add(1.0) * torch.tensor(
        [1.0, -0.5, 0.25], device="cuda")
    all_, few = ssm().quantize_fp8(x), ssm().quantize_fp8(x[-1000:])
    for name in ("q", "scale"):
        assert torch.equal(all_[name][-1000:].view(torch.uint8), few[name].view(torch.uint8))
    peak, scale = x[:, :1].double(), all_["scale"].double()
    # (a quotient in 32 bits: half a step)
    assert bool(((scale * 448 - peak).abs() <= 2.0 ** -24 * peak).all())
    for c, code in enumerate((448.0, -224.0, 112.0)):
        assert bool((all_["q"][:, c].float() == code).all())


def test_refusals_of_shared_memory():
    """Outputs and workspaces over the weight or another tensor of the call, and scales of a wrong number of axes."""
    r = Rand(83)
    x, w, dy = r(1, 256), r(256), r(1, 256)
    n, g, mm = ssm().add_norm_fwd, ssm().add_norm_bwd, ssm().matmul_fp8
    q, s, b = r.codes(6, 256), r.scales(6, 2), r.codes(300, 256)
    for f in (lambda: n(x, w, y=w[None]), lambda: n(x, w, residual_out=w[None]), lambda: n(x, w, y_dtype=F8, y_scale=w[None, 2:4]),
              lambda: g(x, w, dy, dx=w[None]), lambda: g(x, w, dy, dresidual=w[None]), lambda: g(x, w, dy, workspace=w),
              lambda: g(x, w, dy, workspace=dy.view(torch.uint8)), lambda: mm(q, s, b, s[0]), lambda: mm(q, s, b, s[0, 0])):
        with pytest.raises(ValueError):
            f()
