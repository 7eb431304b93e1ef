"""Whole-number inputs of the products with 4-bit weights, whose sums fp32 holds exactly
in any order, and the float64 results to compare with, bit for bit after one rounding.

Scales are powers of two, zero points whole numbers. Every partial sum (of x (128 + q) and
(128 + zero) x over a group, of the groups, of a token's choices) is then a multiple of a
power of two, and `held` checks for the inputs at hand that its magnitude stays below 2^24
such units, whatever the order; a hidden value below 2^16 is two bf16 terms."""
import torch

from tests import _plain_q4 as Q


def held(magnitude, unit):
    """Sums of at most these magnitudes, in multiples of unit, are exact in fp32."""
    assert float(magnitude.max()) < 2.0 ** 24 * unit, float(magnitude.max()) / unit
    return True


def _ints(g, shape, most, device):
    return torch.randint(-most, most + 1, shape, generator=g, device=device, dtype=torch.int32)


def weights(g, shape, group, zero, low, device):
    """(packed, scale, zero points or None, values): scales 2^low and 2^(low + 1). Values
    about as often below 0 as above it, so that sums stay small beside their terms."""
    *lead, K = shape
    q = torch.randint(1, 16, shape, generator=g, device=device, dtype=torch.uint8)
    q *= torch.randint(0, 64, shape, generator=g, device=device, dtype=torch.uint8) > 0
    data = Q.pack(q)
    sc = 2.0 ** (low + torch.randint(0, 2, (*lead, K // group), generator=g, device=device))
    sc = sc.to(torch.bfloat16)
    zp = None
    if zero:
        zp = torch.randint(0, 16, sc.shape, generator=g, device=device).to(torch.bfloat16)
    return data, sc, zp, Q.values(data, sc, zp, group)


def groups_held(x, group):
    """Sums of a group before its scale: x (128 + q) and (128 + zero) x."""
    return held(x.abs().reshape(*x.shape[:-1], -1, group).sum(-1) * (143 + 143), 1.0)


def linear_case(g, N, K, M, group, zero, bias, residual, device="cuda"):
    s = dict(group=group)
    s["x"] = _ints(g, (N, K), 3, device).to(torch.bfloat16)
    s["W"] = weights(g, (M, K), group, zero, -1, device)
    s["b"] = _ints(g, (M,), 100, device).float() if bias else None
    s["r"] = _ints(g, (N, M), 100, device).to(torch.bfloat16) if residual else None
    return s


def linear(s, act):
    """out of a case in float64."""
    x, W = s["x"].double(), s["W"][3]
    groups_held(x, s["group"])
    held(x.abs().sum(1) * float(W.abs().max()) + 200, 0.5)
    y = x @ W.t()
    if s["b"] is not None:
        y = y + s["b"].double()
    if act == "relu":
        y = y.clamp(min=0)
    return y if s["r"] is None else y + s["r"].double()


def experts_case(g, N, d, E, k, d_ff, group, zero, bias, odd, device="cuda"):
    """odd: ids that repeat within a token and ids outside [0, E); token 0 has none."""
    s = dict(group=group, E=E)
    x = _ints(g, (N, d), 1, device) * _ints(g, (N, d), 1, device)
    # (fewer of them in wide layers, whose sums of about d_ff sqrt(d) have to stay in 24 bits)
    x *= torch.rand((N, d), generator=g, device=device) < min(1.0, 6e9 / (float(d_ff) ** 2 * d))
    s["x"] = x.to(torch.bfloat16)
    s["up"] = weights(g, (E, d_ff, d), group, zero, 0, device)
    s["down"] = weights(g, (E, d, d_ff), group, zero, -1, device)
    s["b_up"] = _ints(g, (E, d_ff), 20, device).float() if bias else None
    s["b_down"] = _ints(g, (E, d), 100, device).float() if bias else None
    if odd:
        idx = torch.randint(0, E, (N, k), generator=g, device=device)
        out = torch.tensor([-1, E, 2 ** 31 - 1, -(2 ** 31)], device=device)
        pick = torch.randint(0, 32, (N, k), generator=g, device=device)
        idx = torch.where(pick < 4, out[pick.clamp(max=3)], idx)
        idx[0] = out[torch.arange(k, device=device) % 4]
    else:
        idx = torch.rand((N, E), generator=g, device=device).topk(k, dim=1).indices
    s["idx"] = idx.int()
    s["gate"] = 2.0 ** torch.randint(-1, 1, (N, k), generator=g, device=device).float()
    return s


def experts(s):
    """out of a case in float64 (ReLU)."""
    x, E, group = s["x"].double(), s["E"], s["group"]
    groups_held(x, group)
    out, size = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        up, down = s["up"][3][e], s["down"][3][e]
        held(x[t].abs().sum(1) * float(up.abs().max()) + 20, 1.0)
        h = x[t] @ up.t()
        if s["b_up"] is not None:
            h = h + s["b_up"][e].double()
        h = h.clamp(min=0)
        assert float(h.max()) < 2.0 ** 16
        groups_held(h, group)
        y, m = h @ down.t(), h @ down.abs().t()
        if s["b_down"] is not None:
            y, m = y + s["b_down"][e].double(), m + 100
        held(m, 0.5)
        g = s["gate"][t, j].double()[:, None]
        out.index_add_(0, t, g * y)
        size.index_add_(0, t, g * m)
    held(size, 0.25)
    return out
