"""The 64-bit references of the packed operators (packed_ref.py): their gradients against central differences, and the
recurrence against a state carried over a cut."""
import pytest
import torch

import packed_ref as R

F = torch.float64


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, dtype=F)


def differences(f, leaf, loss_grads, n=6, eps=1e-5):
    """Central differences of the loss in a few entries of ``leaf``: (index, difference)."""
    flat = leaf.view(-1)
    pick = torch.linspace(0, flat.numel() - 1, min(n, flat.numel())).long().tolist()
    out = []
    for i in pick:
        v = float(flat[i])
        flat[i] = v + eps
        up = f()
        flat[i] = v - eps
        down = f()
        flat[i] = v
        out.append((i, (up - down) / (2 * eps)))
    return out


def held(grad, diffs):
    # a central difference with step 1e-5 of a loss of size L errs by about 1e-16 L / 1e-5 and by 1e-10 times its third
    # derivative: 1e-6 of the largest gradient leaves room for both
    g = grad.reshape(-1)
    scale = max(1.0, float(g.abs().max()))
    for i, d in diffs:
        assert abs(float(g[i]) - d) <= 1e-6 * scale, (i, float(g[i]), d)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("K", [1, 2, 4])
def test_conv_gradients(K, act):
    g = torch.Generator().manual_seed(K)
    cu = [0, 5, 5, 6, 8]
    x, w, b, first = rnd(g, 9, 3), rnd(g, 3, K), rnd(g, 3), rnd(g, 4, 3, K - 1)
    du, dl = rnd(g, 9, 3), rnd(g, 4, 3, K - 1)

    def loss():
        _, u, last = R.conv(x, w, b, cu, first, act)
        return float((u[:8] * du[:8]).sum() + (last * dl).sum())

    got = R.conv_grads(x, w, b, cu, first, du, dl, act)
    for k, leaf in (("dx", x), ("dweight", w), ("dbias", b)) + ((("dstate", first),) if K > 1 else ()):
        held(got[k], differences(loss, leaf, None))


@pytest.mark.parametrize("zoh", [False, True])
@pytest.mark.parametrize("softplus", [False, True])
def test_ssd_gradients(zoh, softplus):
    g = torch.Generator().manual_seed(3)
    T, H, P, G, N, cu = 8, 4, 2, 2, 3, [0, 4, 4, 5, 8]
    x, B, C, first = rnd(g, T, H, P), rnd(g, T, G, N), rnd(g, T, G, N), rnd(g, 4, H, P, N)
    dt, bias, D = rnd(g, T, H), rnd(g, H), rnd(g, H)
    if not softplus:
        dt, bias = dt.abs() * 0.3, None
    A = -torch.exp(rnd(g, H))
    dy, dl = rnd(g, T, H, P), rnd(g, 4, H, P, N)

    def loss():
        y, last, _ = R.ssd(x, dt, A, B, C, bias, D, cu, first, softplus, zoh)
        return float((y * dy).sum() + (last * dl).sum())

    got = R.ssd_grads(x, dt, A, B, C, bias, D, cu, first, dy, dl, softplus, zoh)
    for k, leaf in (("dx", x), ("ddt", dt), ("dA", A), ("dB", B), ("dC", C), ("dDskip", D), ("dstate", first)) + \
            ((("ddt_bias", bias),) if bias is not None else ()):
        held(got[k], differences(loss, leaf, None))


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate", [None, True, False])
def test_norm_gradients(gate, center):
    g = torch.Generator().manual_seed(5)
    x, w, b, dy = rnd(g, 3, 12), rnd(g, 12), rnd(g, 12), rnd(g, 3, 12)
    z = None if gate is None else rnd(g, 3, 12)

    def loss():
        return float((R.norm(x, w, b, z, 2, 1e-3, bool(gate), center) * dy).sum())

    got = R.norm_grads(x, w, b, z, 2, 1e-3, bool(gate), center, dy)
    for k, leaf in (("dx", x), ("dweight", w), ("dbias", b)) + ((("dz", z),) if z is not None else ()):
        held(got[k], differences(loss, leaf, None))


def test_states_carry_over_a_cut():
    g = torch.Generator().manual_seed(7)
    T, H, P, N = 9, 2, 2, 3
    x, B, C = rnd(g, T, H, P), rnd(g, T, 1, N), rnd(g, T, 1, N)
    dt, A, first = rnd(g, T, H), -torch.exp(rnd(g, H)), rnd(g, 1, H, P, N)
    y, last, _ = R.ssd(x, dt, A, B, C, None, None, [0, T], first)
    y1, mid, _ = R.ssd(x[:4], dt[:4], A, B[:4], C[:4], None, None, [0, 4], first)
    y2, end, _ = R.ssd(x[4:], dt[4:], A, B[4:], C[4:], None, None, [0, 5], mid)
    assert torch.allclose(torch.cat([y1, y2]), y, rtol=1e-13, atol=1e-13) and torch.allclose(end, last, rtol=1e-13)
    w, cx = rnd(g, 4, 3), rnd(g, T, 4)
    f = rnd(g, 1, 4, 2)
    _, u, lw = R.conv(cx, w, None, [0, T], f)
    _, u1, m = R.conv(cx[:1], w, None, [0, 1], f)
    _, u2, e = R.conv(cx[1:], w, None, [0, T - 1], m)
    assert torch.allclose(torch.cat([u1, u2]), u, rtol=1e-13, atol=1e-13) and torch.equal(e, lw)
