"""moe_linear and moe_linear_backward against their float64 forms: the skinny
path (1 to 64 rows), both tile shapes, ranges of the reduction, widths that end
inside a tile or a K-step, every activation, bias, residual and gradient type."""
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


def _randn(torch, shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# N, K, M, act, bias, residual: rows around the skinny limits and the tiles'
# edges, K around the K-steps (32, 64) and shorter than one, M around 16 and 128
SHAPES = [
    (1, 8, 8, "gelu", True, True), (1, 768, 520, "none", False, False),
    (3, 40, 24, "relu", True, False), (16, 1000, 264, "gelu", True, True),
    (17, 264, 136, "none", True, True), (32, 4104, 72, "gelu", False, False),
    (33, 72, 2056, "relu", True, True), (64, 512, 640, "gelu", True, False),
    (65, 8, 8, "none", True, True), (65, 712, 1000, "gelu", True, True),
    (127, 64, 128, "relu", False, True), (130, 2056, 136, "gelu", True, False),
    (257, 1544, 776, "none", True, True), (1000, 200, 3000, "gelu", True, True),
    (3500, 136, 3592, "relu", True, True), (4097, 520, 3080, "none", False, False),
    # few rows past what the skinny kernel takes, and its half tiles' limits
    (1, 4104, 4360, "gelu", True, True), (9, 4104, 4360, "none", True, False),
    (40, 2056, 1544, "relu", True, True), (64, 4104, 1032, "gelu", False, True),
    (8, 264, 4088, "gelu", True, True), (8, 264, 4096, "relu", True, False),
    (5, 8, 40, "none", False, True), (8, 72, 16, "gelu", True, False),
    # a last round of 256x256 tiles in halves (of 4 rows the lower one is empty),
    # and ranges of the reduction that put two workgroups on a CU
    (4100, 72, 4104, "gelu", True, True), (4612, 200, 4104, "none", True, True),
    (2100, 14344, 1032, "gelu", True, True),
]


@pytest.mark.parametrize("N,K,M,act,bias,residual", SHAPES)
def test_forward(torch_mod, N, K, M, act, bias, residual):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    G.say(f"[linear] N={N} K={K} M={M} {act} bias={bias} residual={residual}")
    x, W = _randn(torch, (N, K), bf, 1), _randn(torch, (M, K), bf, 2, K ** -0.5)
    b = _randn(torch, (M,), torch.float32, 3, 0.5) if bias else None
    r = _randn(torch, (N, M), bf, 4) if residual else None
    # a guard row after the output: nothing past the last row is written
    buf = torch.full((N + 1, M), 7.0, dtype=bf, device="cuda")
    out, z = B.linear(x, W, b, act=act, residual=r, out=buf[:N], keep_z=True)
    torch.cuda.synchronize()
    y, z64, ey, ez = P.linear(x, W, b, act, r)
    P.close(out, y, P.stored(y, ey, bf), "out")
    P.close(z, z64, P.stored(z64, ez, bf), "z")
    assert bool((buf[N] == 7.0).all())
    # without z, and over the residual's buffer: the same bits
    if r is not None:
        r2 = r.clone()
        B.linear(x, W, b, act=act, residual=r2, out=r2)
        assert torch.equal(r2, out)
    else:
        assert torch.equal(B.linear(x, W, b, act=act)[0], out)


BACKWARD = [
    (1, 8, 8, "gelu"), (1, 768, 520, "none"), (5, 200, 136, "relu"), (63, 64, 128, "gelu"),
    (64, 1032, 72, "gelu"), (65, 72, 264, "none"), (127, 136, 1000, "relu"),
    (200, 712, 520, "gelu"), (1031, 264, 2056, "gelu"), (2047, 1000, 136, "none"),
    (3600, 3592, 136, "relu"), (3333, 3080, 3336, "gelu"),
    # weight gradients of at most 64 rows, over several K-steps
    (129, 8, 8, "none"), (300, 264, 56, "gelu"), (2000, 72, 64, "relu"), (640, 1000, 40, "none"),
    # halves of the last round in dx and in dW, ranges with two workgroups a CU in dW
    (4100, 4104, 72, "gelu"), (72, 4104, 4104, "relu"), (15000, 1032, 2056, "none"),
]


@pytest.mark.parametrize("grads", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M,act", BACKWARD)
def test_backward(torch_mod, N, K, M, act, grads):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    dt = torch.float32 if grads == "f32" else bf
    G.say(f"[linear backward] N={N} K={K} M={M} {act} {grads}")
    x, W = _randn(torch, (N, K), bf, 1), _randn(torch, (M, K), bf, 2, K ** -0.5)
    z = _randn(torch, (N, M), bf, 3) if act != "none" else None
    dout = _randn(torch, (N, M), bf, 4)
    dx, dW, db = B.linear_backward(x, W, z, dout, act=act, dx_dtype=dt, dW_dtype=dt)
    torch.cuda.synchronize()
    ref = P.linear_backward(x, W, z, dout, act)
    P.close(dx, ref["dx"][0], P.stored(*ref["dx"], dt), "dx")
    P.close(dW, ref["dW"][0], P.stored(*ref["dW"], dt), "dW")
    P.close(db, ref["db"][0], P.stored(*ref["db"], torch.float32), "db")
    # each gradient alone: the same bits
    only = B.linear_backward(x, W, z, dout, act=act, bias=False, need_dx=False, dW_dtype=dt)
    assert only[0] is None and only[2] is None and torch.equal(only[1], dW)
    only = B.linear_backward(x, W, z, dout, act=act, bias=False, need_dW=False, dx_dtype=dt)
    assert torch.equal(only[0], dx)
    only = B.linear_backward(x, W, z, dout, act=act, need_dx=False, need_dW=False)
    assert torch.equal(only[2], db)


def test_infinities_stay_in_their_rows(torch_mod):
    """A row of x with an infinity or a NaN makes its own output row not
    finite and no other; ReLU keeps a NaN; GELU of -inf is 0."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    bf = torch.bfloat16
    for N in (20, 200):
        K, M = 136, 264
        x, W = _randn(torch, (N, K), bf, 1), _randn(torch, (M, K), bf, 2)
        W = W.abs() + 0.125
        x[3, 7], x[4, 9], x[5, 0] = float("inf"), float("nan"), float("-inf")
        for act in ("relu", "gelu"):
            out, _ = B.linear(x, W, act=act)
            assert bool(torch.isinf(out[3]).all()) and bool(torch.isnan(out[4]).all())
            assert not bool(out[5].any())
            rest = [i for i in range(N) if i not in (3, 4, 5)]
            assert bool(torch.isfinite(out[rest]).all())
        # an infinite gradient where ReLU is off gives 0, not NaN
        z = torch.full((N, M), -1.0, dtype=bf, device="cuda")
        dout = torch.full((N, M), float("inf"), dtype=bf, device="cuda")
        _, _, db = B.linear_backward(x, W, z, dout, act="relu", need_dx=False, need_dW=False)
        assert not bool(db.any())


def test_no_rows_and_leading_dims(torch_mod):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    bf = torch.bfloat16
    W = _randn(torch, (24, 16), bf, 1)
    x = torch.empty((0, 16), dtype=bf, device="cuda")
    out, z = B.linear(x, W, act="relu", keep_z=True)
    assert out.shape == (0, 24)
    dx, dW, db = B.linear_backward(x, W, z, out, act="relu", dW_dtype=bf)
    assert dx.shape == (0, 16) and not bool(dW.any()) and not bool(db.any())
    x3 = _randn(torch, (5, 20, 16), bf, 2)
    out3, _ = B.linear(x3, W, residual=None)
    assert out3.shape == (5, 20, 24)
    assert torch.equal(out3.reshape(100, 24), B.linear(x3.reshape(100, 16), W)[0])


def test_gradient_against_differences(torch_mod):
    """Directional derivatives of the float64 forward against the kernel's
    gradients: dz is rounded to bf16 (2^-8 each, independent), so a projection
    on a random direction holds to 2^-8 of the norms' product."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    N, K, M = 70, 48, 56
    x, W = _randn(torch, (N, K), bf, 1), _randn(torch, (M, K), bf, 2, 0.15)
    b = _randn(torch, (M,), torch.float32, 3)
    c = _randn(torch, (N, M), bf, 4)
    # z as the backward reads it: to bf16, 2^-8 of slope's change (at most 0.8)
    _, z = B.linear(x, W, b, act="gelu", keep_z=True)
    dx, dW, db = B.linear_backward(x, W, z, c, act="gelu")
    f = lambda x, W, b: float((P.act(x @ W.t() + b, "gelu") * c.double()).sum())  # noqa: E731
    args0 = [x.double(), W.double(), b.double()]
    for i, g in enumerate((dx, dW, db)):
        for seed in range(3):
            v = _randn(torch, g.shape, torch.float32, 20 + seed).double()
            hi, lo = list(args0), list(args0)
            hi[i], lo[i] = args0[i] + 1e-5 * v, args0[i] - 1e-5 * v
            want = (f(*hi) - f(*lo)) / 2e-5
            got = float((g.double() * v).sum())
            assert abs(got - want) <= 2.0 ** -8 * float(g.double().norm() * v.norm()), (i, got, want)


def test_offsets_past_32_bits(torch_mod):
    """More than 2^31 elements of z, out and dout: the first and last rows, and
    gradients of a dout that is zero but for some of those rows."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    N, K, M = 262150, 64, 8200
    rows = torch.tensor([0, 1, 777, 131073, N - 130, N - 2, N - 1], device="cuda")
    x, W = _randn(torch, (N, K), bf, 1), _randn(torch, (M, K), bf, 2, K ** -0.5)
    b = _randn(torch, (M,), torch.float32, 3)
    out, z = B.linear(x, W, b, act="gelu", keep_z=True)
    torch.cuda.synchronize()
    y, z64, ey, ez = P.linear(x[rows], W, b, "gelu", None)
    P.close(out[rows], y, P.stored(y, ey, bf), "out")
    P.close(z[rows], z64, P.stored(z64, ez, bf), "z")
    dout = out.zero_()
    dout[rows] = _randn(torch, (len(rows), M), bf, 4)
    G.say("[linear] past 32 bits: backward")
    dx, dW, db = B.linear_backward(x, W, z, dout, act="gelu")
    torch.cuda.synchronize()
    ref = P.linear_backward(x[rows], W, z[rows], dout[rows], "gelu")
    P.close(dx[rows], ref["dx"][0], P.stored(*ref["dx"], torch.float32), "dx")
    P.close(dW, ref["dW"][0], P.stored(*ref["dW"], torch.float32), "dW")
    P.close(db, ref["db"][0], P.stored(*ref["db"], torch.float32), "db")
    dx[rows] = 0
    assert not bool(dx.any())
