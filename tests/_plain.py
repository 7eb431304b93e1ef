"""Float64 forms of the operators around the layer, with the elementwise error
bounds of the fp32 kernels beside them (torch float64 on the tensors' device).

Bounds count, for sums of n products accumulated in fp32 in any order,
gamma(n) = n 2^-24 per term of the sum of magnitudes (2^-23 on the matrix
cores, whose accumulation may truncate), half a step for each rounding to a
stored type, and 1.5e-7 for the erf formula of GELU."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative
ERF = 1.5e-7


def gamma(n, ulp=2.0 ** -23):
    return (n + 4) * ulp


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    return torch.ones_like(z)


def act_error(z, ez, name):
    """Error of the activation of z given an error ez of z: slope at most 1.13,
    the erf formula, and a few fp32 operations."""
    if name == "none":
        return ez
    e = 1.13 * ez
    if name == "gelu":
        e = e + (ERF + 2.0 ** -21) * z.abs()
    return e


def stored(y, e, dtype):
    """Bound of a value y known to e, stored in dtype (with the smallest
    normal's step, for values that underflow)."""
    return e + U[dtype] * (y.abs() + e) + 2.0 ** -126


def close(got, want, tol, what=""):
    """Elementwise |got - want| <= tol."""
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bad = ~((g - want).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{g[i].item()} for {want[i].item()} (bound {tol[i].item():.3g})")


def linear(x, W, b, name, r):
    """(out, z) and their bounds before storage."""
    x, W = x.double(), W.double()
    z = x @ W.t()
    ez = gamma(x.shape[1]) * (x.abs() @ W.abs().t())
    if b is not None:
        z = z + b.double()
        ez = ez + 2.0 ** -23 * (z.abs() + b.double().abs())
    y = act(z, name)
    ey = act_error(z, ez, name)
    if r is not None:
        y = y + r.double()
        ey = ey + 2.0 ** -23 * (y.abs() + r.double().abs())
    return y, z, ey, ez


def linear_backward(x, W, z, dout, name):
    """dx, dW, db and their bounds before storage."""
    x, W, g = x.double(), W.double(), dout.double()
    dz, edz = g, torch.zeros_like(g)
    if name != "none":
        s = act_grad(z.double(), name)
        dz = g * s
        # slope of GELU: the erf formula and a few operations of values below 2
        edz = g.abs() * (ERF + 2.0 ** -20) if name == "gelu" else edz
    e16 = edz + (0 if name == "none" else U[torch.bfloat16]) * (dz.abs() + edz)
    N, M = dz.shape
    az = dz.abs() + e16
    return dict(dx=(dz @ W, e16 @ W.abs() + gamma(M) * (az @ W.abs())),
                dW=(dz.t() @ x, e16.t() @ x.abs() + gamma(N) * (az.t() @ x.abs())),
                db=(dz.sum(0), edz.sum(0) + gamma(N) * (dz.abs() + edz).sum(0)))


def layer_norm(h, w, b, eps):
    """out, mean, rstd and their bounds. Sums run over at most 64 sequential
    fp32 additions per level of the reduction."""
    h, w = h.double(), w.double()
    g = gamma(64, 2.0 ** -24)
    mean = h.mean(1, keepdim=True)
    c = h - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    em = g * h.abs().mean(1, keepdim=True) + 2.0 ** -24 * mean.abs()
    ec = em + 2.0 ** -23 * c.abs()
    ev = (2 * c.abs() * ec + ec * ec).mean(1, keepdim=True) + g * (c.abs() + ec).pow(2).mean(
        1, keepdim=True)
    er = rstd * (ev / (var + eps) + 2.0 ** -21)
    y = c * rstd * w
    ey = w.abs() * ((c.abs() + ec) * er + ec * rstd) + 2.0 ** -22 * y.abs()
    if b is not None:
        y = y + b.double()
        ey = ey + 2.0 ** -23 * (y.abs() + b.double().abs())
    return y, mean[:, 0], rstd[:, 0], ey, em[:, 0], er[:, 0]


def layer_norm_backward(h, w, mean, rstd, dout, dres):
    """dx, dw, db and their bounds for the given mean and rstd."""
    h, w, dy = h.double(), w.double(), dout.double()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    N, d = h.shape
    g0 = gamma(64, 2.0 ** -24)
    xh = (h - m) * r
    ex = 2.0 ** -22 * xh.abs()
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    e1 = g0 * g.abs().mean(1, keepdim=True)
    e2 = (g0 + 2.0 ** -21) * (g * xh).abs().mean(1, keepdim=True)
    edx = r * (2.0 ** -22 * g.abs() + e1 + xh.abs() * e2 + ex * m2.abs()
               + 2.0 ** -21 * (g.abs() + m1.abs() + (xh * m2).abs()))
    if dres is not None:
        dx = dx + dres.double()
        edx = edx + 2.0 ** -23 * (dx.abs() + dres.double().abs())
    gn = gamma(N, 2.0 ** -24)
    return dict(dx=(dx, edx),
                dw=((dy * xh).sum(0), ((gn + 2.0 ** -21) * (dy * xh).abs()).sum(0)),
                db=(dy.sum(0), gn * dy.abs().sum(0)))


def route(x, W_g, noise, k, cf):
    """idx, gate, slot, capacity of the layer's router in float64 (ties to the
    lower id; slots in (choice, token) order)."""
    s = x.double() @ W_g.double().t()
    if noise is not None:
        s = s + noise.double()
    N, E = s.shape
    top, idx = torch.sort(s, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    gate = torch.softmax(top, dim=1)
    C = math.ceil(cf * (k * N) / E)
    seen = [0] * E
    slot = torch.full((N, k), -1, dtype=torch.int64)
    ids = idx.cpu()
    for j in range(k):
        for t in range(N):
            e = int(ids[t, j])
            if seen[e] < C:
                slot[t, j] = seen[e]
            seen[e] += 1
    return idx, gate, slot.to(x.device), C, torch.tensor(seen)


def few(x, W_up, W_down, b_up, b_down, name, idx, gate, slot, rounded_h):
    """out of the layer for the given routing, and its bound before storage.
    rounded_h: relative error of a kept hidden value."""
    x = x.double()
    N, d = x.shape
    d_ff = W_up.shape[1]
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    for e in sorted({int(v) for v in idx.flatten().tolist()}):
        t, j = ((idx == e) & (slot >= 0)).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        wu, wd = W_up[e].double(), W_down[e].double()
        h, _, eh, _ = linear(x[t], wu, None if b_up is None else b_up[e], name, None)
        eh = eh + rounded_h * (h.abs() + eh)
        y = h @ wd.t()
        ey = eh @ wd.abs().t() + gamma(d_ff) * ((h.abs() + eh) @ wd.abs().t())
        if b_down is not None:
            y = y + b_down[e].double()
            ey = ey + 2.0 ** -23 * (y.abs() + b_down[e].double().abs())
        g = gate[t, j].double()[:, None]
        # gates hold to 1e-5 absolute, sums of choices to a few fp32 steps
        out.index_add_(0, t, g * y)
        err.index_add_(0, t, g * ey + (1e-5 + 2.0 ** -19 * g) * (y.abs() + ey))
    return out, err
