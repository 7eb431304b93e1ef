"""Float64 forms of the products with 4-bit weights, with the elementwise error
bounds of the kernels beside them (bounds as in _plain.py). The kernels
accumulate x (128 + q) and x in fp32 and subtract, so a group's terms count with
the magnitude |x| (143 + 128 + |zero|) scale."""
import torch

from tests import _plain as P


def pack(q):
    """uint8 [.., K] of 4-bit numbers -> [.., K / 2], even column in the low half."""
    return q[..., 0::2] | (q[..., 1::2] << 4)


def weights(g, shape, group, zero, device="cuda"):
    """Seeded 4-bit weights of extents [.., M, K]: packed, scale, zero points or
    None, and their float64 values."""
    *lead, K = shape
    q = torch.randint(0, 16, shape, generator=g, device=device, dtype=torch.uint8)
    sc = (0.25 + torch.rand((*lead, K // group), generator=g, device=device)) / (5 * K ** 0.5)
    sc = sc.to(torch.bfloat16)
    zp = None
    if zero:
        zp = torch.randint(0, 16, sc.shape, generator=g, device=device).to(torch.bfloat16)
    return pack(q), sc, zp, values(pack(q), sc, zp, group)


def values(data, scale, zero, group):
    q = torch.stack((data & 15, data >> 4), dim=-1).reshape(*data.shape[:-1], -1).double()
    z = 8.0 if zero is None else zero.double().repeat_interleave(group, dim=-1)
    return (q - z) * scale.double().repeat_interleave(group, dim=-1)


def magnitude(scale, zero, group):
    """|scale| (143 + 128 + |zero|) of every weight."""
    z = 8.0 if zero is None else zero.double().abs()
    return (scale.double().abs() * (271.0 + z)).repeat_interleave(group, dim=-1)


def product(x, W, mag):
    """x W^T and the bound of its fp32 evaluation."""
    x = x.double()
    return x @ W.t(), P.gamma(x.shape[1]) * (x.abs() @ mag.t())


def linear(x, W, mag, b, name, r):
    z, ez = product(x, W, mag)
    if b is not None:
        z = z + b.double()
        ez = ez + 2.0 ** -23 * (z.abs() + b.double().abs())
    y, ey = P.act(z, name), P.act_error(z, ez, name)
    if r is not None:
        y = y + r.double()
        ey = ey + 2.0 ** -23 * (y.abs() + r.double().abs())
    return y, ey


def experts(x, idx, gate, up, down, group, b_up, b_down, name):
    """out of the routed experts and its bound before storage; up, down: (scale,
    zero, values). A hidden value keeps two bf16 terms: 2^-16 of it."""
    x = x.double()
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(up[2].shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        pick = lambda w: (w[2][e], magnitude(w[0][e], None if w[1] is None else w[1][e], group))  # noqa: E731
        h, eh = linear(x[t], *pick(up), None if b_up is None else b_up[e], name, None)
        eh = eh + 2.0 ** -16 * (h.abs() + eh)
        W, mag = pick(down)
        y = h @ W.t()
        ey = eh @ W.abs().t() + P.gamma(2 * W.shape[1]) * ((h.abs() + eh) @ mag.t())
        if b_down is not None:
            y = y + b_down[e].double()
            ey = ey + 2.0 ** -23 * (y.abs() + b_down[e].double().abs())
        g = gate[t, j].double()[:, None]
        out.index_add_(0, t, g * y)
        err.index_add_(0, t, g.abs() * ey + 2.0 ** -19 * g.abs() * (y.abs() + ey))
    return out, err
