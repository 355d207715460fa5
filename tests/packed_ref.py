"""The packed operators from their definitions in 64 bits, token by token (torch on the CPU): references of the tests."""
import torch

F = torch.float64


def silu(v):
    return v / (1 + torch.exp(-v))


def silu_slope(v):
    s = 1 / (1 + torch.exp(-v))
    return s * (1 + v * (1 - s))


def first_states(S, tail, state, idx, has):
    """State that each sequence starts from."""
    out = torch.zeros((S,) + tail, dtype=F)
    for s in range(S):
        k = s if idx is None else int(idx[s])
        if state is not None and 0 <= k < state.shape[0] and (has is None or bool(has[s])):
            out[s] = state[k].to(F)
    return out


def conv(x, w, b, cu, first, act=True):
    """(pre, u, last windows); rows outside every sequence are zero."""
    T, D = x.shape
    K = w.shape[1]
    S = len(cu) - 1
    pre, last = torch.zeros(T, D, dtype=F), torch.zeros(S, D, K - 1, dtype=F)
    for s in range(S):
        a, e = int(cu[s]), int(cu[s + 1])
        row = torch.cat([first[s].T, x[a:e]])                     # (K - 1 + n, D)
        for t in range(e - a):
            pre[a + t] = (row[t:t + K].T * w).sum(1) + (0 if b is None else b)
        last[s] = row[e - a:].T
    return pre, silu(pre) if act else pre, last


def conv_grads(x, w, b, cu, first, du, dlast, act=True):
    T, D = x.shape
    K = w.shape[1]
    S = len(cu) - 1
    pre, _, _ = conv(x, w, b, cu, first, act)
    dpre = du * (silu_slope(pre) if act else 1)
    dx, dw, db, dfirst = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(D, dtype=F), torch.zeros_like(first)
    for s in range(S):
        a, e = int(cu[s]), int(cu[s + 1])
        row = torch.cat([first[s].T, x[a:e]])
        drow = torch.zeros_like(row)
        for t in range(e - a):
            drow[t:t + K] += dpre[a + t] * w.T
            dw += dpre[a + t][:, None] * row[t:t + K].T
            db += dpre[a + t]
        if dlast is not None:
            drow[e - a:] += dlast[s].T
        dx[a:e] = drow[K - 1:]
        dfirst[s] = drow[:K - 1].T
    return {"dx": dx, "dweight": dw, "dbias": db, "dstate": dfirst}


def steps(dt, bias, A, softplus=True, zoh=False):
    """(u, Delta, a, phi)"""
    u = dt + (0 if bias is None else bias)
    d = torch.nn.functional.softplus(u, threshold=60) if softplus else u
    a = torch.exp(d * A)
    phi = torch.where(A == 0, d, torch.expm1(d * A) / torch.where(A == 0, 1, A)) if zoh else d
    return u, d, a, phi


def ssd(x, dt, A, B, C, bias, D, cu, first, softplus=True, zoh=False, keep=False):
    """(y, last states, y's sum of magnitudes[, every state])"""
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    heads = torch.arange(H) // (H // G)
    _, _, a, phi = steps(dt, bias, A, softplus, zoh)
    y, big = torch.zeros(T, H, P, dtype=F), torch.zeros(T, H, P, dtype=F)
    last = torch.zeros_like(first)
    states = torch.zeros(T, H, P, N, dtype=F) if keep else None
    for s in range(len(cu) - 1):
        S, M = first[s].clone(), first[s].abs()
        for t in range(int(cu[s]), int(cu[s + 1])):
            S = S * a[t][:, None, None] + (phi[t][:, None] * x[t])[:, :, None] * B[t, heads][:, None]
            M = M * a[t][:, None, None] + (phi[t][:, None] * x[t]).abs()[:, :, None] * B[t, heads].abs()[:, None]
            y[t] = (S * C[t, heads][:, None]).sum(-1) + (0 if D is None else D[:, None] * x[t])
            big[t] = (M * C[t, heads].abs()[:, None]).sum(-1) + (0 if D is None else (D[:, None] * x[t]).abs())
            if keep:
                states[t] = S
        last[s] = S
    return (y, last, big, states) if keep else (y, last, big)


def ssd_grads(x, dt, A, B, C, bias, D, cu, first, dy, dlast, softplus=True, zoh=False):
    T, H, P = x.shape
    G = B.shape[1]
    heads = torch.arange(H) // (H // G)
    u, d, a, phi = steps(dt, bias, A, softplus, zoh)
    _, _, _, states = ssd(x, dt, A, B, C, bias, None, cu, first, softplus, zoh, keep=True)
    out = {"dx": torch.zeros_like(x), "dB": torch.zeros_like(B), "dC": torch.zeros_like(C), "dstate": torch.zeros_like(first)}
    dlog, dphi = torch.zeros_like(d), torch.zeros_like(d)
    inside = torch.zeros(T, 1, dtype=F)
    for s in range(len(cu) - 1):
        b0, e0 = int(cu[s]), int(cu[s + 1])
        inside[b0:e0] = 1
        Gs = torch.zeros_like(first[s]) if dlast is None else dlast[s].clone()
        for t in range(e0 - 1, b0 - 1, -1):
            Gs = Gs + dy[t][:, :, None] * C[t, heads][:, None]           # dL / dS_t
            prev = states[t - 1] if t > b0 else first[s]
            GB = (Gs * B[t, heads][:, None]).sum(-1)
            out["dx"][t] = phi[t][:, None] * GB + (0 if D is None else D[:, None] * dy[t])
            out["dB"][t].index_add_(0, heads, (Gs * (phi[t][:, None] * x[t])[:, :, None]).sum(1))
            out["dC"][t].index_add_(0, heads, (states[t] * dy[t][:, :, None]).sum(1))
            dphi[t] = (GB * x[t]).sum(-1)
            dlog[t] = (Gs * prev).sum((1, 2)) * a[t]
            Gs = Gs * a[t][:, None, None]
        out["dstate"][s] = Gs
    if zoh:
        dd = A * dlog + a * dphi
        zero = A == 0
        slope = torch.where(zero, d * d / 2, (d * a - phi) / torch.where(zero, 1, A))     # d phi / dA
        out["dA"] = (d * dlog + slope * dphi).sum(0)
    else:
        dd = A * dlog + dphi
        out["dA"] = (d * dlog).sum(0)
    out["ddt"] = dd / (1 + torch.exp(-u)) if softplus else dd
    out["ddt_bias"] = (out["ddt"] * inside).sum(0)
    out["dDskip"] = (dy * x * inside[:, :, None]).sum((0, 2))
    return out


def norm(x, w, b, z, groups, eps, first, center):
    T, D = x.shape
    h = x * silu(z) if z is not None and first else x
    h = h.reshape(T, groups, -1)
    if center:
        h = h - h.mean(-1, keepdim=True)
    y = (h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)).reshape(T, D) * w
    if b is not None:
        y = y + b
    return y * silu(z) if z is not None and not first else y


def norm_grads(x, w, b, z, groups, eps, first, center, dy):
    T, D = x.shape
    n = D // groups
    gate = None if z is None else silu(z)
    pre = z is not None and first
    h = (x * gate if pre else x).reshape(T, groups, n)
    if center:
        h = h - h.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    nh = (h * r).reshape(T, D)
    line = nh * w + (0 if b is None else b)
    dline = dy * gate if z is not None and not first else dy
    dn = (dline * w).reshape(T, groups, n)
    nn = nh.reshape(T, groups, n)
    dh = dn - nn * (dn * nn).mean(-1, keepdim=True)
    if center:
        dh = dh - dn.mean(-1, keepdim=True)
    dh = (dh * r).reshape(T, D)
    out = {"dx": dh * gate if pre else dh, "dweight": (dline * nh).sum(0), "dbias": dline.sum(0), "dz": None}
    if z is not None:
        out["dz"] = (dh * x if pre else dy * line) * silu_slope(z)
    return out
