"""Products with 4-bit weights against their float64 forms: groups, zero
points, row counts on both sides of every token tile, widths that end inside a
tile or a wave's step, duplicate and invalid ids, and the conversions."""
import pytest

from tests import _gpu as G

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


def _randn(torch, g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


# (N, K, M, group): single groups, K off the 128-wide step, M off every tile,
# token tiles 1, 2 and 4, few and many waves
LINEAR = [(1, 32, 1, 32), (1, 64, 5, 64), (2, 128, 16, 128), (3, 96, 33, 32), (16, 160, 48, 32),
          (17, 192, 31, 64), (5, 320, 100, 64), (32, 1152, 64, 128), (33, 1056, 257, 32),
          (64, 2048, 130, 64), (1, 7168, 2048, 128), (7, 4128, 2050, 32), (48, 4096, 3000, 128),
          (9, 14336, 512, 64), (64, 8064, 35000, 128), (1, 640, 70000, 32)]


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,M,group", LINEAR)
def test_linear(torch_mod, N, K, M, group, zero):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P, _plain_q4 as Q
    G.say(f"[q4 linear] N={N} K={K} M={M} group={group} zero={zero}")
    g = _gen(torch, N + K + M)
    data, sc, zp, W = Q.weights(g, (M, K), group, zero)
    x = _randn(torch, g, (N, K), torch.bfloat16)
    b = _randn(torch, g, (M,), torch.float32) if M % 3 else None
    r = _randn(torch, g, (N, M), torch.bfloat16) if K % 64 == 0 else None
    act = ("none", "relu", "gelu")[(N + M) % 3]
    w = B.Q4(data, sc, zp, group=group)
    out = B.linear_q4(x, w, b, act=act, residual=r)
    torch.cuda.synchronize()
    y, ey = Q.linear(x, W, Q.magnitude(sc, zp, group), b, act, r)
    P.close(out, y, P.stored(y, ey, torch.bfloat16), "out")
    assert torch.equal(B.linear_q4(x, w, b, act=act, residual=r), out)
    if r is not None:   # in place of the residual
        assert torch.equal(B.linear_q4(x, w, b, act=act, residual=r, out=r), out)


# (N, d, E, k, d_ff, group)
EXPERTS = [(1, 32, 1, 1, 32, 32), (1, 128, 4, 2, 256, 128), (2, 96, 5, 3, 160, 32),
           (8, 192, 3, 2, 320, 64), (9, 128, 2, 1, 384, 128), (16, 768, 8, 2, 2048, 32),
           (17, 256, 2, 2, 128, 64), (33, 384, 3, 3, 640, 128), (64, 256, 2, 2, 512, 32),
           (64, 1024, 256, 16, 128, 128), (61, 2048, 32, 8, 1024, 64), (1, 4096, 8, 2, 14336, 128)]


def _layer(torch, g, N, d, E, k, d_ff, group, zero):
    from tests import _plain_q4 as Q
    up = Q.weights(g, (E, d_ff, d), group, zero)
    down = Q.weights(g, (E, d, d_ff), group, zero)
    x = _randn(torch, g, (N, d), torch.bfloat16)
    idx = torch.rand((N, E), generator=g, device="cuda").topk(k, dim=1).indices.int()
    gate = torch.rand((N, k), generator=g, device="cuda") + 0.1
    return x, idx, gate, up, down


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,d,E,k,d_ff,group", EXPERTS)
def test_experts(torch_mod, N, d, E, k, d_ff, group, zero):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P, _plain_q4 as Q
    G.say(f"[q4 experts] N={N} d={d} E={E} k={k} d_ff={d_ff} group={group} zero={zero}")
    g = _gen(torch, N + d + E)
    x, idx, gate, up, down = _layer(torch, g, N, d, E, k, d_ff, group, zero)
    bias = E % 2 == 0
    bu = _randn(torch, g, (E, d_ff), torch.float32) if bias else None
    bd = _randn(torch, g, (E, d), torch.float32) if bias else None
    act = "gelu" if bias else "relu"
    args = (x, idx, gate, B.Q4(*up[:3], group=group), B.Q4(*down[:3], group=group))
    out = B.experts_q4(*args, act=act, b_up=bu, b_down=bd)
    torch.cuda.synchronize()
    y, ey = Q.experts(x, idx, gate, up[1:], down[1:], group, bu, bd, act)
    P.close(out, y, P.stored(y, ey, torch.bfloat16), "out")
    assert torch.equal(B.experts_q4(*args, act=act, b_up=bu, b_down=bd), out)


@pytest.mark.parametrize("N", [1, 5, 40, 64])
def test_duplicate_and_invalid_ids(torch_mod, N):
    """The same id twice in a token counts twice (one expert then has more rows
    than tokens), an id outside [0, E) not at all; a token without a valid id
    gives zeros."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P, _plain_q4 as Q
    d, E, k, d_ff, group = 256, 4, 4, 384, 64
    g = _gen(torch, N)
    x, idx, gate, up, down = _layer(torch, g, N, d, E, k, d_ff, group, True)
    idx[:, 1] = idx[:, 0]
    idx[0] = torch.tensor([3, 3, 3, 3])
    if N > 1:
        idx[1:, :3] = 2
        idx[1] = torch.tensor([-1, 4, 2 ** 31 - 1, -(2 ** 31)])
        idx[2, 3] = 256
    out = B.experts_q4(x, idx, gate, B.Q4(*up[:3], group=group), B.Q4(*down[:3], group=group))
    y, ey = Q.experts(x, idx, gate, up[1:], down[1:], group, None, None, "relu")
    P.close(out, y, P.stored(y, ey, torch.bfloat16), "out")
    if N > 1:
        assert not bool(out[1].any())


def test_values_that_are_not_finite_stay_in_their_row(torch_mod):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain_q4 as Q
    g = _gen(torch, 3)
    data, sc, zp, W = Q.weights(g, (96, 256), 64, False)
    x = _randn(torch, g, (20, 256), torch.bfloat16)
    w = B.Q4(data, sc, zp, group=64)
    want = B.linear_q4(x, w)
    x[3, 7], x[17, 200] = float("nan"), float("inf")
    got = B.linear_q4(x, w)
    for t in range(20):
        if t in (3, 17):
            assert bool(torch.isnan(got[t]).all())
        else:
            assert torch.equal(got[t], want[t])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("shape,group", [((1, 32), 32), ((7, 192), 64), ((3, 5, 256), 128),
                                         ((130, 4096), 32)])
def test_quantize(torch_mod, shape, group, zero, dtype):
    """The format's definition in float64, but for weights within 2^-20 of the
    middle of two steps (the kernel divides in fp32); the values of it are
    exact in fp32 and rounded once in bf16."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain_q4 as Q
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = _gen(torch, len(shape) + group)
    W = _randn(torch, g, shape, dt, 0.05)
    W[..., :group] = 0
    W[..., 0, group:group + 2] = 0
    q = B.quantize_q4(W, group=group, zero=zero)
    torch.cuda.synchronize()
    w = W.double().reshape(*shape[:-1], -1, group)
    hi, lo = w.amax(-1).clamp(min=0), w.amin(-1).clamp(max=0)
    want = (hi - lo) / 15 if zero else torch.maximum(hi, -lo) / 7
    s = q.scale.double()
    # bf16 of the fp32 quotient: half a step and a few fp32 roundings
    assert bool(((s - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want).all())
    live = s > 0
    assert bool((live == (want > 0)).all())
    nibble = torch.stack((q.data & 15, q.data >> 4), dim=-1).reshape(w.shape).double()
    sd = torch.where(live, s, torch.ones_like(s))
    z = torch.full_like(s, 8.0)
    if zero:
        z = q.zero.double()
        e = (z - (-lo / sd).clamp(0, 15)).abs()
        assert bool((e <= 0.5 + 2.0 ** -20).all()) and bool((z == z.round()).all())
    ideal = (w / sd[..., None] + z[..., None]).clamp(0, 15)
    assert bool(((nibble - ideal).abs() <= 0.5 + 2.0 ** -18)[live].all())
    assert bool((nibble == z[..., None])[~live].all())
    value = Q.values(q.data, q.scale, q.zero, group)
    assert torch.equal(B.dequantize_q4(q, dtype=torch.float32).double(), value)
    assert torch.equal(B.dequantize_q4(q), value.to(torch.bfloat16))
