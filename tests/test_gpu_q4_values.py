"""The 4-bit products and conversions at values where bounds of accumulated roundings
would not tell a fault: whole numbers, whose sums are exact in fp32 in any order, over
every form that the kernels take; the distance from float64 in the 2-norm, by row and by
16 columns; the edges of the range."""
import pytest

from tests import _gpu as G
from tests import test_gpu_q4 as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_mod():
    if not G.have_gpu():
        pytest.skip("no HIP device")
    import torch
    from sparse_mixture_experts_20_amd import binding as B
    B.lib()
    return torch


def _gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_whose_range_is_past_fp32(torch_mod, dtype):
    """max - min of a group of finite weights past the largest fp32 number: scale, zero
    point and values as for any other group (scale: half a bf16 step and a few fp32
    roundings; a value half a step of the scale and what the scale's rounding moves, at
    most 15 x 2^-9)."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    W = torch.randn((4, 64), generator=_gen(torch, 1), device="cuda").clamp(-3, 3) * 1e38
    W[:, 0], W[:, 40] = 3e38, -2e38
    W[3] = W[3].abs()         # a range of one sign for comparison
    W = W.to(dt)
    q = B.quantize_q4(W, group=64, zero=True)
    w = W.double()
    hi, lo = w.amax(1).clamp(min=0), w.amin(1).clamp(max=0)
    assert bool((hi - lo > torch.finfo(torch.float32).max)[:3].all())
    want = (hi - lo) / 15
    s = q.scale.double()[:, 0]
    assert bool(((s - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want).all())
    z = q.zero.double()[:, 0]
    assert bool(((z + lo / s).abs() <= 0.5 + 2.0 ** -18).all())
    got = B.dequantize_q4(q, dtype=torch.float32).double()
    assert bool(torch.isfinite(got).all())
    assert bool(((got - w).abs() <= s[:, None] * (1.0 + 15 * 2.0 ** -8)).all())


def _rows_norm(got, want):
    """The largest distance of a row, relative, in the 2-norm."""
    return float(((got.double() - want).norm(dim=1) / want.norm(dim=1)).max())


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", [1, 20, 40])
def test_large_finite_activations(torch_mod, N, group, zero):
    """Activations, and hidden values of the experts, up to the stated range: sum |x| over
    a group just below 2^119. (bf16 output: half a step of 2^-8 at most, fp32 sums on
    top: 2^-16 of the magnitudes.)"""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain_q4 as Q
    K, M = 512, 96
    g = _gen(torch, N + group)
    x = torch.randn((N, K), generator=g, device="cuda")
    big = 2.0 ** 118.99 / float(x.abs().reshape(N, -1, group).sum(2).max())
    x = (x * big).to(torch.bfloat16)
    assert 2.0 ** 118 < float(x.double().abs().reshape(N, -1, group).sum(2).max()) < 2.0 ** 119
    data, sc, zp, W = Q.weights(g, (M, K), group, zero)
    out = B.linear_q4(x, B.Q4(data, sc, zp, group=group))
    assert _rows_norm(out, x.double() @ W.t()) <= 2.0 ** -8
    # the experts: one that leads up to the range and one that leads back
    E, k, d, d_ff = 3, 2, 256, K
    up, down = Q.weights(g, (E, d_ff, d), group, zero), Q.weights(g, (E, d, d_ff), group, zero)
    x = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    h = torch.relu(x.double() @ up[3].reshape(E * d_ff, d).t()).reshape(N, E, -1, group)
    shift = 118 - int(torch.log2(h.sum(3).max()).ceil())
    upv, downv = up[3] * 2.0 ** shift, down[3]
    idx = torch.rand((N, E), generator=g, device="cuda").topk(k, dim=1).indices.int()
    gate = torch.rand((N, k), generator=g, device="cuda") + 0.1
    scale = (up[1].float() * 2.0 ** shift).to(torch.bfloat16)     # (a power of two: exact)
    out = B.experts_q4(x, idx, gate, B.Q4(up[0], scale, up[2], group=group),
                       B.Q4(*down[:3], group=group))
    want = torch.zeros((N, d), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        y = torch.relu(x[t].double() @ upv[e].t()) @ downv[e].t()
        want.index_add_(0, t, gate[t, j].double()[:, None] * y)
    assert bool(torch.isfinite(out).all())
    assert _rows_norm(out, want) <= 2.0 ** -8


# (N, K, M): one, two and four token tiles, one and two weight tiles a wave (two from 4096
# strips of 16 rows on), all of K in one buffer or in two, waves along the rows and along
# K, widths that end inside a step, a tile and a strip. K is cut to a multiple of the group.
LINEAR = [(1, 128, 1), (3, 160, 33), (16, 1152, 257), (7, 7168, 512), (16, 8064, 130),
          (17, 224, 50), (29, 4128, 100), (33, 640, 48), (64, 8064, 200), (48, 2048, 2050),
          (17, 128, 65600), (40, 352, 65600), (64, 1152, 66000), (9, 384, 70000),
          (1, 14336, 2048), (5, 14336, 4096)]


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K,M", LINEAR)
def test_linear_of_whole_numbers(torch_mod, N, K, M, group, zero):
    """out, to the last bit: the float64 result rounded once."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _whole_q4 as H
    K = K // group * group
    G.say(f"[q4 values] linear N={N} K={K} M={M} group={group} zero={zero}")
    s = H.linear_case(_gen(torch, N + K + M), N, K, M, group, zero, M % 3, N % 2)
    w = B.Q4(*s["W"][:3], group=group)
    for act in ("none", "relu"):
        out = B.linear_q4(s["x"], w, s["b"], act=act, residual=s["r"])
        torch.cuda.synchronize()
        assert torch.equal(out, H.linear(s, act).to(torch.bfloat16))


def test_linear_past_2_to_the_31_weights(torch_mod):
    """Rows whose weights lie on both sides of 2^31 and 2^32 of them (whole numbers)."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _whole_q4 as H
    K, M, group = 16384, (1 << 18) + 40, 128
    g = _gen(torch, 4)
    data = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sc = 2.0 ** torch.randint(-1, 1, (M, K // group), generator=g, device="cuda")
    sc = sc.to(torch.bfloat16)
    w = B.Q4(data, sc, group=group)
    some = torch.cat([torch.arange(a, a + 40, device="cuda")
                      for a in (0, (1 << 17) - 20, (1 << 18) - 20, M - 40)])
    for N in (2, 20):
        G.say(f"[q4 values] linear N={N} of {M} x {K} weights")
        x = torch.randint(-3, 4, (N, K), generator=g, device="cuda").to(torch.bfloat16)
        out = B.linear_q4(x, w)
        V = H.Q.values(data[some], sc[some], None, group)
        assert torch.equal(out[:, some], (x.double() @ V.t()).to(torch.bfloat16))


# (N, d, E, k, d_ff), as above for both products; without a plan and with one, rows of an
# expert in one pass and in several, choices added by the last workgroup of a column block
# or (past 4096 workgroups of the down product) by a launch of their own
EXPERTS = [(1, 128, 4, 2, 256), (2, 256, 5, 3, 384), (16, 768, 8, 2, 2048), (6, 512, 3, 3, 4096),
           (5, 4096, 6, 2, 4096), (64, 256, 256, 16, 128), (61, 512, 32, 8, 384),
           (20, 256, 4, 2, 16384), (20, 16384, 4, 2, 256), (64, 128, 8, 2, 8192),
           (64, 8192, 8, 2, 1024), (64, 2048, 256, 16, 128), (4, 8192, 64, 16, 128),
           (33, 384, 3, 3, 640), (30, 384, 4, 2, 1152), (24, 128, 2, 1, 256),
           (3, 14336, 4, 1, 2048), (12, 2048, 3, 1, 14336), (64, 512, 4, 2, 8192)]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,d,E,k,d_ff", EXPERTS)
def test_experts_of_whole_numbers(torch_mod, N, d, E, k, d_ff, group, zero, odd):
    """out, to the last bit; odd: ids that repeat within a token (an expert then has more
    rows than tokens), ids outside [0, E), a token without any."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _whole_q4 as H
    G.say(f"[q4 values] experts N={N} d={d} E={E} k={k} d_ff={d_ff} group={group} zero={zero} "
          f"odd={odd}")
    s = H.experts_case(_gen(torch, N + d + E), N, d, E, k, d_ff, group, zero, E % 2 == 0, odd)
    up, down = (B.Q4(*s[n][:3], group=group) for n in ("up", "down"))
    ws = B.alloc_workspace(B.experts_q4_workspace_size(N, d, E, d_ff, k, group))
    ws.fill_(255)      # (rows of an invalid id are not written, and must not be read)
    for _ in range(2):
        out = B.experts_q4(s["x"], s["idx"], s["gate"], up, down, b_up=s["b_up"],
                           b_down=s["b_down"], workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, H.experts(s).to(torch.bfloat16))


def _far(got, want):
    """The largest distances in the 2-norm, relative: of a row and of 16 columns (of all,
    where there are fewer than 16 either way)."""
    d, w = got.double() - want, want
    rows = d.norm(dim=1) / w.norm(dim=1) if d.shape[1] >= 16 else d.norm() / w.norm()
    n = d.shape[1] // 16 * 16
    far = float(rows.max())
    if n and d.shape[0] >= 16:
        c = d[:, :n].reshape(d.shape[0], -1, 16).norm(dim=(0, 2))
        far = max(far, float((c / w[:, :n].reshape(d.shape[0], -1, 16).norm(dim=(0, 2))).max()))
    return far


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,M,group", T.LINEAR)
def test_linear_distance(torch_mod, N, K, M, group, zero):
    """Half a bf16 step is 2^-8 of a value at most, 2^-9.2 in the mean of many; what fp32
    adds is below 2^-16 of a row. A group of K left out would be sqrt(group / K) of it, 2^-4.4
    at the longest K here, one column of 14336 2^-6.9."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P, _plain_q4 as Q
    g = _gen(torch, N + K + M)
    data, sc, zp, W = Q.weights(g, (M, K), group, zero)
    x = torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16)
    for act in ("none", "gelu"):
        out = B.linear_q4(x, B.Q4(data, sc, zp, group=group), act=act)
        assert _far(out, P.act(x.double() @ W.t(), act)) <= 2.0 ** -8


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,d,E,k,d_ff,group", T.EXPERTS)
def test_experts_distance(torch_mod, N, d, E, k, d_ff, group, zero):
    """As above; the hidden row's 2^-16 adds less than 2^-16 of an output row."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain_q4 as Q
    g = _gen(torch, N + d + E)
    x, idx, gate, up, down = T._layer(torch, g, N, d, E, k, d_ff, group, zero)
    bu = torch.randn((E, d_ff), generator=g, device="cuda")
    bd = torch.randn((E, d), generator=g, device="cuda")
    args = (B.Q4(*up[:3], group=group), B.Q4(*down[:3], group=group))
    for act, biases in (("relu", (None, None)), ("gelu", (bu, bd))):
        out = B.experts_q4(x, idx, gate, *args, act=act, b_up=biases[0], b_down=biases[1])
        want, _ = Q.experts(x, idx, gate, up[1:], down[1:], group, *biases, act)
        assert _far(out, want) <= 2.0 ** -8
