"""moe_forward_few on small whole numbers, where every sum is exact in fp32 in
any order, so that the output has to be the float64 result rounded once: no
bound of accumulated roundings can hide a missing term, row, range or expert.
And the distance from float64 in the 2-norm, where bounds of single elements
are wide."""
import pytest

from tests import _gpu as G
from tests import test_gpu_few as F

pytestmark = pytest.mark.gpu

# Sums of magnitudes up to here are exact in fp32 (half of its 2^24, as the two terms
# of a hidden value may have opposite signs).
EXACT = 2.0 ** 23


@pytest.fixture(scope="module")
def torch_mod():
    if not G.have_gpu():
        pytest.skip("no HIP device")
    import torch
    from sparse_mixture_experts_20_amd import binding as B
    B.lib()
    return torch


def _whole(torch, g, shape, most, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda",
                         dtype=torch.int8).to(dtype)


def _sparse_down(torch, g, E, d, d_ff, dtype):
    """W_down rows of few nonzeros, the last 8 columns (a tail of the reduction)
    and the first always among them."""
    w = _whole(torch, g, (E, d, d_ff), 3, dtype)
    keep = torch.rand((E, d, d_ff), generator=g, device="cuda") < min(1.0, 24.0 / d_ff)
    keep[:, :, -8:] = True
    keep[:, :, 0] = True
    return torch.where(keep, w, torch.zeros_like(w))


def _expected(torch, x, wu, wd, bu, bd, idx, slot, gate, first_term_only=False):
    """The layer in float64, ReLU, and the largest sum of magnitudes in it."""
    out, most = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), 0.0
    mag = torch.zeros_like(out)
    x = x.double()
    for e in sorted({int(v) for v in idx.flatten().tolist()}):
        t, j = ((idx == e) & (slot >= 0)).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        u, w = wu[e].double(), wd[e].double()
        h = (x[t] @ u.t() + bu[e].double()).clamp(min=0)
        most = max(most, float((x[t].abs() @ u.abs().t() + bu[e].double().abs()).max()))
        assert float(h.max()) < 2.0 ** 16     # two bf16 terms hold it
        if first_term_only:
            h = h.to(torch.bfloat16).double()
        g = gate[t, j].double()[:, None]
        out.index_add_(0, t, g * (h @ w.t() + bd[e].double()))
        mag.index_add_(0, t, h @ w.abs().t() + bd[e].double().abs())
    return out, max(most, float(mag.max()))


# N, E, k, d, d_ff, dtype, capacity factor. bf16: 7 E >= N k streams the weights,
# more rows run on tiles; odd rows of fp32 layers; tails of every step size
CASES = [
    (1, 8, 2, 768, 1032, "bf16", 2.0), (5, 40, 2, 264, 520, "bf16", 40.0),
    (8, 40, 2, 72, 264, "bf16", 40.0), (9, 40, 2, 264, 520, "bf16", 40.0),
    (16, 40, 2, 520, 136, "bf16", 40.0), (20, 40, 2, 264, 2056, "bf16", 40.0),
    (33, 40, 2, 136, 520, "bf16", 40.0), (64, 64, 2, 264, 264, "bf16", 64.0),
    (61, 256, 2, 200, 72, "bf16", 1.5), (64, 40, 2, 264, 520, "bf16", 4.0),
    (64, 8, 2, 264, 520, "bf16", 8.0), (40, 4, 2, 1000, 1000, "bf16", 1.0),
    (64, 2, 1, 72, 4104, "bf16", 2.0), (17, 2, 2, 2056, 72, "bf16", 1.0),
    (1, 4, 2, 3, 9, "f32", 8.0), (21, 6, 2, 515, 1021, "f32", 1.0),
    (40, 40, 2, 130, 77, "f32", 40.0), (64, 5, 2, 260, 516, "f32", 5.0),
    (64, 40, 1, 257, 2050, "f32", 40.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_whole_numbers(torch_mod, case):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    N, E, k, d, d_ff, dtype, cf = case
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(N + d)
    G.say(f"[few values] {case}")
    x = _whole(torch, g, (N, d), 31, dt)
    wu = _whole(torch, g, (E, d_ff, d), 31 if d <= 600 else 15, dt)
    wd = _sparse_down(torch, g, E, d, d_ff, dt)
    bu = _whole(torch, g, (E, d_ff), 100, torch.float32)
    bd = _whole(torch, g, (E, d), 100, torch.float32)
    # k equal scores a token (gates 1 / k, exact for 1 and 2), half of the tokens
    # on experts E / 2 and E / 2 + 1
    pick = torch.rand((N, E), generator=g, device="cuda").argsort(1)[:, :k]
    pick[::2] = (E // 2 + torch.arange(k, device="cuda")) % E
    noise = torch.zeros((N, E), device="cuda").scatter_(1, pick, 5.0)
    out, st = B.forward_few(x, torch.zeros((E, d), device="cuda"), noise, wu, wd, k, cf,
                            b_up=bu, b_down=bd)
    torch.cuda.synchronize()
    assert torch.equal(st.idx.long(), pick.sort(1).values)
    assert bool((st.gate == 1.0 / k).all())
    want, most = _expected(torch, x, wu, wd, bu, bd, st.idx.long(), st.slot, st.gate)
    assert most < EXACT
    assert torch.equal(out, want.to(dt))
    # what the check is for would show: no output, and a hidden row of one term
    assert bool((want != 0).double().mean() > 0.5) or cf < 4.0
    if dtype == "bf16":
        one, _ = _expected(torch, x, wu, wd, bu, bd, st.idx.long(), st.slot, st.gate, True)
        assert not torch.equal(one.to(dt), want.to(dt))


@pytest.mark.parametrize("N", [3, 64])
def test_whole_numbers_past_32_bits(torch_mod, N):
    """Weights of more than 2^31 elements, every token on the last expert: on
    the streaming products and on the tiles."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    E, d, d_ff = 8, 16384, 16392
    bf = torch.bfloat16
    assert E * d * d_ff > 2 ** 31 and (N * 1 > 7 * E) == (N == 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    wu = torch.empty((E, d_ff, d), dtype=bf, device="cuda")
    wd = torch.empty((E, d, d_ff), dtype=bf, device="cuda")
    for e in range(E):   # no expert's weights are another's
        wu[e] = _whole(torch, g, (d_ff, d), 2, bf)
        wd[e] = _sparse_down(torch, g, 1, d, d_ff, bf)[0]
    x = _whole(torch, g, (N, d), 7, bf)
    noise = torch.zeros((N, E), device="cuda")
    noise[:, E - 1] = 9.0
    bu, bd = torch.zeros((E, d_ff), device="cuda"), torch.zeros((E, d), device="cuda")
    G.say(f"[few values] past 32 bits, N={N}")
    out, st = B.forward_few(x, torch.zeros((E, d), device="cuda"), noise, wu, wd, 1, 8.0)
    torch.cuda.synchronize()
    assert bool((st.idx == E - 1).all()) and bool((st.slot >= 0).all())
    want, most = _expected(torch, x, wu, wd, bu, bd, st.idx.long(), st.slot, st.gate)
    assert most < EXACT
    assert torch.equal(out, want.to(bf))
    other, _ = _expected(torch, x, wu, wd, bu, bd, st.idx.long() - 1, st.slot, st.gate)
    assert float((other.to(bf) == want.to(bf)).double().mean()) < 0.1


@pytest.mark.parametrize("case", F.CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_distance_in_the_2_norm(torch_mod, case):
    """For the routing and gates of the call: the output's own rounding (2^-8 or
    2^-24 of each element), the two terms of a bf16 layer's hidden row (2^-16)
    and fp32 sums, at most 256 dependent additions of 2^-24 each per product."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    wl, dev = F._layer(torch, *case)
    c = wl.cfg
    out, st = B.forward_few(dev["x"], dev["W_g"], dev["noise"], dev["W_up"], dev["W_down"], c.k,
                            c.cf, act=c.act, b_up=dev["b_up"], b_down=dev["b_down"])
    torch.cuda.synchronize()
    y, _ = P.few(dev["x"], dev["W_up"], dev["W_down"], dev["b_up"], dev["b_down"], c.act,
                 st.idx.long(), st.gate, st.slot, 0.0)
    limit = 2 * 2.0 ** -16 + (2.0 ** -8 + 2.0 ** -16 if c.dtype == "bf16" else 2.0 ** -24)
    err, size = float((out.double() - y).norm()), float(y.norm())
    G.say(f"[few values] {case}: {err / max(size, 1e-30):.2e} of {limit:.2e}")
    assert err <= limit * size
