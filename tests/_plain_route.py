"""Float64 forms of the routing and its backward, with error bounds.

Inputs are whole multiples of powers of two whose products and sums fp32 holds
exactly, so the scores s are exact and p carries only the roundings of exp,
sums over the experts (tree of at most 12 levels), and divisions: at most 2^-20
relative, which `REL` is."""
import torch

from tests import _plain as P

REL = 2.0 ** -20


def inputs(g, N, d, E, dtype, sigma=False, device="cuda"):
    """x (whole numbers up to 3), W_g and noise (multiples of 2^-10): scores of
    standard deviation about 1, exact in fp32 (their units stay below 2^24)."""
    span = max(1, min(512, int(1024 / (2 * d ** 0.5)) * 2))
    x = torch.randint(-3, 4, (N, d), generator=g, device=device).to(dtype)
    w = torch.randint(-span, span + 1, (E, d), generator=g, device=device).float() / 1024
    assert 3 * span * d + 4096 < 2 ** 24
    noise = None
    if sigma:
        noise = torch.randint(-1024, 1025, (N, E), generator=g, device=device).float() / 1024
    return x, w, noise


def scores(x, W_g, noise, score):
    s = x.double() @ W_g.double().t()
    if noise is not None:
        s = s + noise.double()
    return torch.sigmoid(s) if score == "sigmoid" else torch.softmax(s, dim=1)


def choice(p, bias, k, groups=1, keep=0, best=1):
    """ids in float64 and the rows whose choice fp32 may take otherwise (a gap
    above 0 below the bound of c: equal values stay equal in fp32)."""
    N, E = p.shape
    keep = keep or groups
    c = p if bias is None else p + bias.double()
    tol = REL * p + (0.0 if bias is None else 2.0 ** -23 * c.abs())
    tol = 2 * tol.amax(1)
    near = torch.zeros(N, dtype=torch.bool, device=p.device)

    def close(v):
        gap = v[:, :-1] - v[:, 1:]
        return (gap > 0) & (gap < 2 * tol[:, None])
    if keep < groups:
        size = E // groups
        s = torch.sort(c.reshape(N, groups, size), dim=2, descending=True).values
        s = s[:, :, :min(best, size)].sum(2)
        top, order = torch.sort(s, dim=1, descending=True, stable=True)
        near |= close(top[:, keep - 1:keep + 1])[:, 0]
        ok = torch.zeros((N, groups), dtype=torch.bool, device=p.device)
        ok.scatter_(1, order[:, :keep], True)
        c = c.masked_fill(~ok.repeat_interleave(size, dim=1), -float("inf"))
    top, order = torch.sort(c, dim=1, descending=True, stable=True)
    near |= close(top[:, :min(k + 1, E)]).any(1)
    return order[:, :k], near


def gates(p, idx, renorm, scale):
    g = p.gather(1, idx.long())
    if renorm:
        g = g / g.sum(1, keepdim=True)
    return scale * g


def backward(x, W_g, idx, p, dgate, dp, dres, score, renorm, scale):
    """dx, dW_g of the definition for the given p, and their bounds before
    storage (for products as accurate as fp32 ones)."""
    p, dg, W, x = p.double(), dgate.double(), W_g.double(), x.double()
    N, E = p.shape
    ok = (idx >= 0) & (idx < E)
    i = idx.long().clamp(0, E - 1)
    pc = torch.where(ok, p.gather(1, i), torch.zeros_like(dg))
    dg = torch.where(ok, dg, torch.zeros_like(dg))
    if renorm:
        S = pc.sum(1, keepdim=True)
        u = pc / S
        dc = scale / S * (dg - (u * dg).sum(1, keepdim=True))
        mag = scale / S * (dg.abs() + (u * dg.abs()).sum(1, keepdim=True))
        dc, mag = torch.nan_to_num(dc), torch.nan_to_num(mag)
    else:
        dc, mag = scale * dg, scale * dg.abs()
    dc, mag = torch.where(ok, dc, 0 * dc), torch.where(ok, mag, 0 * mag)
    full = torch.zeros_like(p).scatter_add_(1, i, dc)
    fmag = torch.zeros_like(p).scatter_add_(1, i, mag)
    if dp is not None:
        full, fmag = full + dp.double(), fmag + dp.double().abs()
    if score == "sigmoid":
        ds = full * p * (1 - p)
        eds = REL * fmag * p * (1 - p)
    else:
        dot = (full * p).sum(1, keepdim=True)
        ds = p * (full - dot)
        eds = REL * p * (fmag + (fmag * p).sum(1, keepdim=True))
    dW = ds.t() @ x
    eW = eds.t() @ x.abs() + P.gamma(3 * N) * ((ds.abs() + eds).t() @ x.abs())
    dx = ds @ W
    ex = eds @ W.abs() + P.gamma(6 * E) * ((ds.abs() + eds) @ W.abs())
    if dres is not None:
        dx = dx + dres.double()
        ex = ex + 2.0 ** -23 * (dx.abs() + dres.double().abs())
    sixteen = 2.0 ** -14 * (ds.abs() @ W.abs())   # operands of 16 bits: twice 2^-15
    return dict(dx=(dx, ex), dW=(dW, eW), ds=ds, sixteen=sixteen)
