"""The Mamba-2 block's operators over packed tokens, as they are measured: the causal convolution, the state space scan
(SSD) and the gated group norm, for prompts of uneven length, for single tokens and for training.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math
import random

import torch

own = False

Q = 64          # tokens per chunk of the plain form of the scan
P = 64          # head width


# ---------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the convolution over a batch of uneven prompts, some of them continued, in the 2.7B layer (5120 + 2 x 128 channels)
        dict(name="conv.prompt", op="conv", way="prompt", dtype="bf16", tokens=16384, seqs=11, cut=1, heads=80, groups=1, dstate=128, width=4),
        # one new token for each of 256 requests, same layer
        dict(name="conv.tokens", op="conv", way="tokens", dtype="bf16", tokens=256, seqs=256, cut=0, heads=80, groups=1, dstate=128, width=4),
        # gradients over packed documents, same layer
        dict(name="conv.train", op="conv", way="train", dtype="bf16", tokens=8191, seqs=5, cut=2, heads=80, groups=1, dstate=128, width=4),
        # the scan over a batch of uneven prompts, 2.7B layer
        dict(name="ssd.prompt", op="ssd", way="prompt", dtype="bf16", tokens=16384, seqs=11, cut=1, heads=80, groups=1, dstate=128, zoh=False),
        # one very long prompt in the 130M layer (1536 channels = 24 heads)
        dict(name="ssd.prompt.long", op="ssd", way="prompt", dtype="bf16", tokens=65537, seqs=1, cut=0, heads=24, groups=1, dstate=128, zoh=False),
        # one new token for each of 256 requests, 2.7B layer
        dict(name="ssd.tokens", op="ssd", way="tokens", dtype="bf16", tokens=256, seqs=256, cut=0, heads=80, groups=1, dstate=128, zoh=False),
        # one request alone, 130M layer: latency
        dict(name="ssd.tokens.one", op="ssd", way="tokens", dtype="bf16", tokens=1, seqs=1, cut=0, heads=24, groups=1, dstate=128, zoh=False),
        # gradients over packed documents, 2.7B layer
        dict(name="ssd.train", op="ssd", way="train", dtype="bf16", tokens=16384, seqs=6, cut=3, heads=80, groups=1, dstate=128, zoh=False, carry=False),
        # a small training batch, two groups, zero-order hold, states carried in and out
        dict(name="ssd.train.small", op="ssd", way="train", dtype="bf16", tokens=1999, seqs=3, cut=4, heads=24, groups=2, dstate=64, zoh=True, carry=True),
        # the norm behind the scan over the prompts' tokens, gate first, one group, 2.7B layer
        dict(name="norm.prompt", op="norm", way="prompt", dtype="bf16", tokens=16384, dim=5120, groups=1, gate=True, gate_first=True, center=False),
        # the norm of single tokens in 32 bits, mean taken off, eight groups, gate behind it
        dict(name="norm.tokens", op="norm", way="prompt", dtype="f32", tokens=256, dim=1536, groups=8, gate=True, gate_first=False, center=True),
        # its gradients, 2.7B layer, eight groups
        dict(name="norm.train", op="norm", way="train", dtype="bf16", tokens=8191, dim=5120, groups=8, gate=True, gate_first=True, center=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "ssd", "ssd", "norm"])
    way = rng.choice(["prompt", "train"] if op == "norm" else ["prompt", "tokens", "train"])
    if op == "norm":
        groups = rng.choice([1, 1, 2, 5, 8])
        return dict(op=op, way=way, dtype=rng.choice(["bf16", "bf16", "f32"]), tokens=_log(rng, 1, 8000), dim=groups * _log(rng, 60, 5120 // groups),
                    groups=groups, gate=rng.random() < 0.8, gate_first=rng.random() < 0.7, center=rng.random() < 0.3)
    groups = rng.choice([1, 1, 1, 2, 4])
    heads = groups * _log(rng, 2, 80 // groups)
    case = dict(op=op, way=way, dtype="bf16" if op == "ssd" else rng.choice(["bf16", "bf16", "f32"]), heads=heads, groups=groups,
                dstate=rng.choice([64, 128, 128, 256]) if heads <= 40 else rng.choice([64, 128]))
    if op == "conv":
        case["width"] = rng.choice([2, 3, 4, 4])
    else:
        case["zoh"] = rng.random() < 0.3
    if way == "tokens":
        case["tokens"] = case["seqs"] = _log(rng, 1, 256)
        case["cut"] = 0
    else:
        case["tokens"] = _log(rng, 1, 16000 if op == "conv" else 6000)
        case["seqs"] = rng.randint(1, min(12, case["tokens"]))
        case["cut"] = rng.randint(1, 10 ** 6)
    if op == "ssd" and way == "train":
        case["carry"] = rng.random() < 0.5
    return case


def _lens(case):
    """Lengths of the sequences: uneven pieces of the tokens, from one token up."""
    t, s = case["tokens"], case["seqs"]
    if s == t:
        return [1] * t
    cuts = sorted(random.Random(case["cut"]).sample(range(1, t), s - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _channels(case):
    return case["heads"] * P + 2 * case["groups"] * case["dstate"]


# ---------------------------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def logu(lo, hi, *shape):
        return torch.exp(torch.rand(*shape, generator=gen, device="cuda") * (math.log(hi) - math.log(lo)) + math.log(lo))

    s = {"case": case}
    T = case["tokens"]
    if case["op"] == "norm":
        D = case["dim"]
        s["x"] = randn(T, D, dtype=dt)
        # the gate is the first part of the layer's projected input: rows further apart than they are long
        s["z"] = randn(T, 2 * D + 256, dtype=dt)[:, :D] if case["gate"] else None
        s["weight"] = 1 + randn(D, scale=0.1)
        s["bias"] = randn(D, scale=0.1) if case["center"] else None
        if case["way"] == "train":
            s["dy"] = randn(T, D, dtype=dt)
        return s
    H, G, N, S = case["heads"], case["groups"], case["dstate"], case["seqs"]
    C = _channels(case)
    lens = _lens(case)
    s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    slots = S + 3
    s["idx"] = torch.randperm(slots, generator=gen, device="cuda")[:S].to(torch.int32)
    s["has"] = torch.rand(S, generator=gen, device="cuda") < 0.5
    # the projected input of a layer holds gate, convolved channels and step sizes side by side
    proj = randn(T, H * P + C + H, dtype=dt)
    if case["op"] == "conv":
        K = case["width"]
        s["x"] = proj[:, H * P:H * P + C]
        s["w"] = randn(C, K, scale=1 / math.sqrt(K))
        s["b"] = randn(C, scale=0.2)
        if case["way"] == "train":
            s["du"] = randn(T, C, dtype=dt)
        else:
            s["state"] = randn(slots, C, K - 1)
        return s
    conv = randn(T, C, dtype=torch.float32)
    conv = (conv * torch.sigmoid(conv)).to(dt)      # what the convolution hands on
    s["x"] = conv[:, :H * P].view(T, H, P)
    s["B"] = conv[:, H * P:H * P + G * N].view(T, G, N)
    s["C"] = conv[:, H * P + G * N:].view(T, G, N)
    s["dt"] = proj[:, H * P + C:]
    s["A"] = -logu(1.0, 16.0, H)
    step = logu(1e-3, 1e-1, H)
    s["bias"] = step + torch.log(-torch.expm1(-step))   # softplus(bias) = step
    s["D"] = 1 + randn(H, scale=0.1)
    if case["way"] != "train":
        s["state"] = randn(slots, H, P, N, scale=0.3)
    else:
        s["dy"] = randn(T, H, P, dtype=dt)
        s["h0"] = randn(S, H, P, N, scale=0.3) if case["carry"] else None
        s["dh"] = randn(S, H, P, N, scale=0.3) if case["carry"] else None
    return s


# ---------------------------------------------------------------------------------------------------------------
# the operators

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "norm":
        return _plain_norm(state, case)
    if case["op"] == "conv":
        return _plain_conv(state, case)
    return _plain_ssd(state, case)


def _own(s, case):
    import selective_state_space_57_amd as ssm
    if case["op"] == "norm":
        kw = dict(bias=s["bias"], z=s["z"], groups=case["groups"], gate_first=case["gate_first"], center=case["center"])
        if case["way"] == "prompt":
            return ssm.gated_norm_fwd(s["x"], s["weight"], **kw)
        g = ssm.gated_norm_bwd(s["x"], s["weight"], s["dy"], **kw)
        return {k: g[k] for k in _norm_grads(s)}
    if case["op"] == "conv":
        if case["way"] == "prompt":
            u = ssm.conv1d_packed_fwd(s["x"], s["w"], s["cu"], s["b"], state=s["state"], state_out=s["state"],
                                      state_idx=s["idx"], has_state=s["has"])
            return u, s["state"]
        if case["way"] == "tokens":
            return ssm.conv1d_slot_update(s["state"], s["x"], s["w"], s["b"], state_idx=s["idx"]), s["state"]
        g = ssm.conv1d_packed_bwd(s["x"], s["w"], s["du"], s["cu"], s["b"])
        return {k: g[k] for k in ("dx", "dweight", "dbias")}
    disc = ssm.ZOH if case["zoh"] else ssm.EULER_B
    if case["way"] == "prompt":
        y = ssm.ssd_packed_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], s["bias"], s["D"], state=s["state"],
                               state_out=s["state"], state_idx=s["idx"], has_state=s["has"], disc=disc)
        return y, s["state"]
    if case["way"] == "tokens":
        y = ssm.ssd_slot_update(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["bias"], s["D"],
                                state_idx=s["idx"], disc=disc)
        return y, s["state"]
    g = ssm.ssd_packed_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], s["cu"], s["bias"], s["D"],
                           state=s["h0"], dstate_out=s["dh"], disc=disc)
    return {k: g[k] for k in _ssd_grads(case)}


def _ssd_grads(case):
    return ("dx", "ddt", "dA", "dB", "dC", "dDskip", "ddt_bias") + (("dstate",) if case["carry"] else ())


def _norm_grads(s):
    return ("dx", "dweight") + (("dz",) if s["z"] is not None else ()) + (("dbias",) if s["bias"] is not None else ())


def _silu(v):
    return v * torch.sigmoid(v)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


# -- norm

def _norm(x, z, w, b, case):
    T, D = x.shape
    g = case["groups"]
    h = x * _silu(z) if z is not None and case["gate_first"] else x
    h = h.view(T, g, D // g)
    if case["center"]:
        h = h - h.mean(-1, keepdim=True)
    y = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5)).view(T, D) * w
    if b is not None:
        y = y + b
    return y * _silu(z) if z is not None and not case["gate_first"] else y


def _plain_norm(s, case):
    f = {k: None if s[k] is None else s[k].float() for k in ("x", "z", "weight", "bias")}
    if case["way"] == "prompt":
        return _norm(f["x"], f["z"], f["weight"], f["bias"], case).to(s["x"].dtype)
    names = {"dx": "x", "dz": "z", "dweight": "weight", "dbias": "bias"}
    keys = _norm_grads(s)
    leaves = [f[names[k]].requires_grad_() for k in keys]
    y = _norm(f["x"], f["z"], f["weight"], f["bias"], case)
    got = torch.autograd.grad(y, leaves, s["dy"].float())
    return {k: v.to(s[names[k]].dtype) for k, v in zip(keys, got)}


# -- convolution

def _places(cu, T):
    """Sequence and position in it of every token."""
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    return seq, t - cu[seq].long()


def _window(x, state, seq, pos, K, back):
    """The input `back` tokens earlier: the sequence's own, or the window that came with it (zeros without one)."""
    inside = pos >= back
    before = state[seq, :, (K - 1 + pos - back).clamp(0, max(K - 2, 0))] if state is not None else torch.zeros((), device=x.device)
    return torch.where(inside[:, None], x[(torch.arange(len(pos), device=x.device) - back).clamp(min=0)], before) if back else x


def _conv(x, w, b, state, seq, pos):
    K = w.shape[1]
    taps = [w[:, k] * _window(x, state, seq, pos, K, K - 1 - k) for k in range(K)]
    return _silu(sum(taps) + b)


def _plain_conv(s, case):
    K, dt = case["width"], s["x"].dtype
    x = s["x"].float()
    if case["way"] == "tokens":
        win = torch.cat([s["state"][s["idx"].long()], x[:, :, None]], 2)
        s["state"][s["idx"].long()] = win[:, :, 1:]
        return _silu((win * s["w"]).sum(2) + s["b"]).to(dt), s["state"]
    seq, pos = _places(s["cu"], case["tokens"])
    if case["way"] == "prompt":
        first = s["state"][s["idx"].long()] * s["has"][:, None, None]
        u = _conv(x, s["w"], s["b"], first, seq, pos).to(dt)
        end = s["cu"][1:].long()
        n = end - s["cu"][:-1].long()
        at = n[:, None] - (K - 1) + torch.arange(K - 1, device=n.device)        # position of each kept input
        new = x[(s["cu"][:-1].long()[:, None] + at).clamp(min=0)].transpose(1, 2)
        old = torch.gather(first, 2, (at + K - 1).clamp(0, max(K - 2, 0))[:, None].expand(-1, x.shape[1], -1))
        s["state"][s["idx"].long()] = torch.where((at >= 0)[:, None], new, old)
        return u, s["state"]
    w, b = s["w"].clone().requires_grad_(), s["b"].clone().requires_grad_()
    x.requires_grad_()
    gx, gw, gb = torch.autograd.grad(_conv(x, w, b, None, seq, pos), (x, w, b), s["du"].float())
    return {"dx": gx.to(dt), "dweight": gw, "dbias": gb}


# -- scan

def _steps(dt, bias, A, zoh):
    """Step size, logarithm of the decay and weight of the new input, of every token and head."""
    delta = _softplus(dt + bias)
    log_a = delta * A
    return log_a, torch.expm1(log_a) / A if zoh else delta


def _scan(x, dt, A, B, C, bias, D, first, cu, zoh):
    """Masked products inside chunks of Q tokens, and one product over the chunks of a sequence between them."""
    T, H, _ = x.shape
    G = B.shape[1]
    seq, pos = _places(cu, T)
    n = (cu[1:] - cu[:-1]).long()
    chunks = (n + Q - 1) // Q
    before = chunks.cumsum(0) - chunks
    nc = T // Q + len(n)                                   # room for all chunks: the last ones may hold nothing
    at = (before[seq] + pos // Q) * Q + pos % Q            # each token's place among the chunks
    log_a, phi = _steps(dt, bias, A, zoh)

    def lay(v):
        return torch.zeros(nc * Q, *v.shape[1:], device=v.device).index_copy(0, at, v).view(nc, Q, *v.shape[1:])

    xs, Bs, Cs = lay(x).transpose(1, 2), lay(B).transpose(1, 2), lay(C).transpose(1, 2)         # (nc, H or G, Q, .)
    la, ph = lay(log_a).transpose(1, 2), lay(phi).transpose(1, 2)                               # (nc, H, Q)
    cum = la.double().cumsum(2)
    total = cum[:, :, -1]
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    mask = torch.where(low, cum[:, :, :, None] - cum[:, :, None], -math.inf).exp().float()
    heads = torch.arange(H, device=x.device) // (H // G)
    scores = torch.matmul(Cs, Bs.transpose(2, 3))[:, heads]
    y = torch.matmul(scores * mask * ph[:, :, None], xs)
    weight = (total[:, :, None] - cum).exp().float() * ph
    ends = torch.matmul((xs * weight[..., None]).transpose(2, 3), Bs[:, heads])                 # (nc, H, P, N)
    chunk = torch.arange(nc, device=x.device)
    owner = torch.searchsorted(chunks.cumsum(0), chunk, right=True)
    run_ = total.cumsum(0)
    prev = run_ - total
    same = (owner[:, None] == owner[None]) & (chunk[:, None] > chunk[None])
    far = torch.where(same[None], prev.T[:, :, None] - run_.T[:, None], -math.inf).exp().float()  # (H, nc, nc)
    carried = torch.matmul(far, ends.transpose(0, 1).reshape(H, nc, -1)).view(H, nc, *ends.shape[2:]).transpose(0, 1)
    own_, start = owner.clamp(max=len(n) - 1), before.clamp(max=nc - 1)
    live = (owner < len(n))[:, None]
    if first is not None:
        drop = torch.where(live, prev - prev[start[own_]], -math.inf).exp().float()
        carried = carried + drop[:, :, None, None] * first[own_]
    y = y + torch.matmul(Cs[:, heads], carried.transpose(2, 3)) * cum.exp().float()[..., None]
    y = y.transpose(1, 2).reshape(nc * Q, H, -1)[at] + D[:, None] * x
    last = (before + chunks - 1).clamp(min=0)
    return y, carried[last] * total[last].exp().float()[:, :, None, None] + ends[last]


def _plain_ssd(s, case):
    zoh, dt = case["zoh"], s["x"].dtype
    f = {k: s[k].float() for k in ("x", "dt", "B", "C")}
    if case["way"] == "tokens":
        heads = torch.arange(case["heads"], device=s["x"].device) // (case["heads"] // case["groups"])
        log_a, phi = _steps(f["dt"], s["bias"], s["A"], zoh)
        at = s["idx"].long()
        new = s["state"][at] * log_a.exp()[..., None, None] + (phi[..., None] * f["x"])[..., None] * f["B"][:, heads, None]
        s["state"][at] = new
        return ((new * f["C"][:, heads, None]).sum(-1) + s["D"][:, None] * f["x"]).to(dt), s["state"]
    if case["way"] == "prompt":
        first = s["state"][s["idx"].long()] * s["has"][:, None, None, None]
        y, last = _scan(f["x"], f["dt"], s["A"], f["B"], f["C"], s["bias"], s["D"], first, s["cu"], zoh)
        s["state"][s["idx"].long()] = last
        return y.to(dt), s["state"]
    names = dict(dx="x", ddt="dt", dA="A", dB="B", dC="C", dDskip="D", ddt_bias="bias", dstate="h0")
    f.update(A=s["A"].clone(), D=s["D"].clone(), bias=s["bias"].clone(), h0=None if s["h0"] is None else s["h0"].clone())
    keys = _ssd_grads(case)
    leaves = [f[names[k]].requires_grad_() for k in keys]
    y, last = _scan(f["x"], f["dt"], f["A"], f["B"], f["C"], f["bias"], f["D"], f["h0"], s["cu"], zoh)
    outs, grads = ([y], [s["dy"].float()]) if s["dh"] is None else ([y, last], [s["dy"].float(), s["dh"]])
    got = torch.autograd.grad(outs, leaves, grads)
    return {k: v.to(s[names[k]].dtype) for k, v in zip(keys, got)}


# ---------------------------------------------------------------------------------------------------------------
# cost

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    T = case["tokens"]
    if case["op"] == "norm":
        n = T * case["dim"]
        arrays = (3 if case["gate"] else 2) + (0 if case["way"] == "prompt" else 2 if case["gate"] else 1)
        return {"bytes": n * e * arrays + 8 * case["dim"], "flops": n * (8 if case["way"] == "prompt" else 20)}
    H, G, N, S, C = case["heads"], case["groups"], case["dstate"], case["seqs"], _channels(case)
    if case["op"] == "conv":
        K = case["width"]
        if case["way"] == "train":
            return {"bytes": 3 * T * C * e + 2 * C * (K + 1) * 4, "flops": T * C * (6 * K + 8)}
        return {"bytes": 2 * T * C * e + 2 * S * C * (K - 1) * 4, "flops": T * C * (2 * K + 4)}
    heads, sides, entries = T * H * P, T * G * N, S * H * P * N * 4
    if case["way"] == "train":
        return {"bytes": (3 * heads + 4 * sides + 2 * T * H) * e + (3 * entries if case["carry"] else 0), "flops": 12 * heads * N}
    return {"bytes": (2 * heads + 2 * sides + T * H) * e + 2 * entries, "flops": 4 * heads * N}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "norm":
        return _exact_norm(d, case)
    lens = _lens(case)
    idx, has = s["idx"].tolist(), s["has"].tolist()
    return _exact_conv(d, case, lens, idx, has) if case["op"] == "conv" else _exact_ssd(d, case, lens, idx, has)


def _exact_norm(d, case):
    x, z, w, b = d["x"], d["z"], d["weight"], d["bias"]
    g = case["groups"]
    T, D = x.shape
    n = D // g
    sig = None if z is None else 1 / (1 + torch.exp(-z))
    gate = None if z is None else z * sig
    slope = None if z is None else sig * (1 + z * (1 - sig))
    first = z is not None and case["gate_first"]
    h = (x * gate if first else x).reshape(T, g, n)
    mean = h.sum(-1, keepdim=True) / n if case["center"] else 0.0
    r = 1 / ((h - mean).square().sum(-1, keepdim=True) / n + 1e-5).sqrt()
    unit = (h - mean) * r
    flat = unit.reshape(T, D)
    line = flat * w + (0 if b is None else b)
    if case["way"] == "prompt":
        return line if z is None or first else line * gate
    up = d["dy"]
    dline = up if z is None or first else up * gate
    dunit = (dline * w).reshape(T, g, n)
    dh = dunit - unit * (dunit * unit).sum(-1, keepdim=True) / n
    if case["center"]:
        dh = dh - dunit.sum(-1, keepdim=True) / n
    dh = (dh * r).reshape(T, D)
    out = {"dx": dh * gate if first else dh, "dweight": (dline * flat).sum(0)}
    if z is not None:
        out["dz"] = (dh * x if first else up * line) * slope
    if b is not None:
        out["dbias"] = dline.sum(0)
    return out


def _exact_conv(d, case, lens, idx, has):
    K, x, w, b = case["width"], d["x"], d["w"], d["b"]
    us, dxs, o = [], [], 0
    gw, gb = torch.zeros_like(w), torch.zeros_like(b)
    tokens = case["way"] == "tokens"
    for k, n in enumerate(lens):
        head = d["state"][idx[k]].T if "state" in d and (tokens or has[k]) else torch.zeros(K - 1, x.shape[1], dtype=x.dtype, device=x.device)
        row = torch.cat([head, x[o:o + n]])
        pre = b + sum(row[j:j + n] * w[:, j] for j in range(K))
        sig = 1 / (1 + torch.exp(-pre))
        us.append(pre * sig)
        if case["way"] == "train":
            dpre = d["du"][o:o + n] * sig * (1 + pre * (1 - sig))
            drow = torch.zeros_like(row)
            for j in range(K):
                drow[j:j + n] += dpre * w[:, j]
                gw[:, j] += (dpre * row[j:j + n]).sum(0)
            gb += dpre.sum(0)
            dxs.append(drow[K - 1:])
        else:
            d["state"][idx[k]] = row[n:].T
        o += n
    if case["way"] == "train":
        return {"dx": torch.cat(dxs), "dweight": gw, "dbias": gb}
    return torch.cat(us), d["state"]


def _exact_ssd(d, case, lens, idx, has):
    H, G, N = case["heads"], case["groups"], case["dstate"]
    train = case["way"] == "train"
    T = case["tokens"]
    u = d["dt"] + d["bias"]
    delta = torch.where(u > 0, u + torch.log1p(torch.exp(-u.abs())), torch.log1p(torch.exp(-u.abs())))
    a = torch.exp(delta * d["A"])
    phi = torch.expm1(delta * d["A"]) / d["A"] if case["zoh"] else delta
    if case["way"] == "tokens":
        gh = torch.arange(H, device=a.device) // (H // G)
        at = torch.tensor(idx, device=a.device)
        new = torch.einsum("bh,bhpn->bhpn", a, d["state"][at]) + torch.einsum("bh,bhp,bhn->bhpn", phi, d["x"], d["B"][:, gh])
        d["state"][at] = new
        return torch.einsum("bhpn,bhn->bhp", new, d["C"][:, gh]) + d["D"][:, None] * d["x"], d["state"]
    y = torch.empty_like(d["x"])
    out = {"dx": torch.empty_like(d["x"]), "ddt": torch.empty_like(d["dt"]), "dA": torch.zeros_like(d["A"]), "dB": torch.zeros_like(d["B"]),
           "dC": torch.zeros_like(d["C"])} if train else None
    longest = max(lens)
    per = H // G
    slab = max(1, min(per, int(16e9 / 8 / (longest + 1) / P / N))) if train else per      # heads at once
    dlog = torch.zeros_like(delta)
    dphi = torch.zeros_like(delta)
    dstate = torch.zeros(len(lens), H, P, N, dtype=a.dtype, device=a.device)
    for h0 in [h for g in range(G) for h in range(g * per, (g + 1) * per, slab)]:
        g = h0 // per
        h1 = min(h0 + slab, (g + 1) * per)
        o = 0
        for k, n in enumerate(lens):
            sl = (slice(o, o + n), slice(h0, h1))
            x, Bk, Ck = d["x"][sl], d["B"][o:o + n, g], d["C"][o:o + n, g]
            ak, px = a[sl], phi[sl][..., None] * x
            if train:
                S0 = d["h0"][k, h0:h1] if d["h0"] is not None else torch.zeros(h1 - h0, P, N, dtype=a.dtype, device=a.device)
                Ss = torch.empty(n + 1, h1 - h0, P, N, dtype=a.dtype, device=a.device)
                Ss[0] = S0
                for t in range(n):
                    torch.mul(Ss[t], ak[t][:, None, None], out=Ss[t + 1])
                    Ss[t + 1].addcmul_(px[t][..., None], Bk[t])
                Gs = torch.empty(n, h1 - h0, P, N, dtype=a.dtype, device=a.device)
                last = d["dh"][k, h0:h1] if d["dh"] is not None else torch.zeros_like(S0)
                dy = d["dy"][sl]
                for t in range(n - 1, -1, -1):
                    if t == n - 1:
                        Gs[t] = last
                    else:
                        torch.mul(Gs[t + 1], ak[t + 1][:, None, None], out=Gs[t])
                    Gs[t].addcmul_(dy[t][..., None], Ck[t])
                dstate[k, h0:h1] = Gs[0] * ak[0][:, None, None]
                GB = (Gs * Bk[:, None, None]).sum(-1)
                out["dx"][sl] = phi[sl][..., None] * GB + d["D"][h0:h1, None] * dy
                dphi[sl] = (GB * x).sum(-1)
                del GB
                out["dB"][o:o + n, g] += torch.matmul(px.reshape(n, 1, -1), Gs.view(n, -1, N)).view(n, N)
                out["dC"][o:o + n, g] += torch.matmul(dy.reshape(n, 1, -1), Ss[1:].reshape(n, -1, N)).view(n, N)
                Gs.mul_(Ss[:-1])
                dlog[sl] = Gs.sum((2, 3)) * ak
                del Gs, Ss
            else:
                S = d["state"][idx[k], h0:h1] * (1.0 if has[k] else 0.0)
                for t in range(n):
                    S = S * ak[t][:, None, None]
                    S.addcmul_(px[t][..., None], Bk[t])
                    y[o + t, h0:h1] = torch.mv(S.view(-1, N), Ck[t]).view(-1, P)
                d["state"][idx[k], h0:h1] = S
            o += n
    if not train:
        return y + d["D"][:, None] * d["x"], d["state"]
    A, dec = d["A"], a
    ddelta = A * dlog + (dec * dphi if case["zoh"] else dphi)
    out["dA"] = (delta * dlog).sum(0) + ((delta * dec - phi) / A * dphi).sum(0) * (1.0 if case["zoh"] else 0.0)
    out["ddt"] = ddelta / (1 + torch.exp(-u))
    out["ddt_bias"] = out["ddt"].sum(0)
    out["dDskip"] = (d["dy"] * d["x"]).sum((0, 2))
    if case["carry"]:
        out["dstate"] = dstate
    return out
