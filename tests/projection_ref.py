"""64-bit definitions of the operators at a block's ends, written from the formulas: e4m3 values with a scale for each block
of 128, the residual's addition with the root mean square norm and its gradient, the product of 8-bit operands."""
import torch

BLOCK, TOP, LEAST = 128, 448.0, 2.0 ** -100


def up(n, m):
    return (n + m - 1) // m * m


def spread(scale, rows, shape):
    """The scale of every entry of a matrix of this shape; blocks of `rows` rows and 128 columns."""
    return scale.repeat_interleave(rows, 0)[:shape[0]].repeat_interleave(BLOCK, 1)[:, :shape[1]]


def magnitudes(x, rows):
    """The largest magnitude of every block of `rows` rows and 128 columns."""
    T, D = x.shape
    v = torch.zeros(up(T, rows), up(D, BLOCK), dtype=torch.float64, device=x.device)
    v[:T, :D] = x.double().abs()
    return v.view(v.shape[0] // rows, rows, -1, BLOCK).amax((1, 3))


def scales(x, rows):
    """fp32 scales: the largest magnitude over 448, rounded once (of an fp32 value's quotient, rounding to 53 bits first does
    not change what 24 bits give)."""
    return (magnitudes(x, rows).clamp(min=LEAST) / TOP).float()


def half_step(v):
    """Half the distance between the e4m3 values around v: 3 bits behind the first one, at least 2^-9 apart."""
    return 0.5 * torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)


def values(q, scale, rows):
    """What codes and scales stand for."""
    return q.double() * spread(scale.double(), rows, q.shape)


def product(a, sa, b, sb, b_rows):
    """out, and the sums of magnitudes of what is added: a (M, K), b (N, K) codes."""
    x, y = values(a, sa, 1), values(b, sb, b_rows)
    return x @ y.T, x.abs() @ y.abs().T


def add_norm(x, residual, weight, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    r = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    return h, h * r * weight.double()


def add_norm_grads(h, weight, dy, dh, eps):
    """dsum, dweight and the sums of magnitudes of what is added to each."""
    h, w, dy = h.double(), weight.double(), dy.double()
    r = (h.square().mean(1, keepdim=True) + eps).rsqrt()
    dn, u = dy * w, h * r
    d = 0 if dh is None else dh.double()
    ds = r * (dn - u * (dn * u).mean(1, keepdim=True)) + d
    size = r * (dn.abs() + u.abs() * (dn * u).abs().mean(1, keepdim=True)) + (0 if dh is None else d.abs())
    return ds, (dy * u).sum(0), size, (dy * u).abs().sum(0)
