"""moe_linear and moe_linear_backward at values where bounds of accumulated
roundings would not tell a fault: small whole numbers, whose sums are exact in
fp32 in any order, over the shapes of tests/test_gpu_linear.py; the distance
from float64 in the 2-norm; NaN; the largest extents."""
import pytest

from tests import _gpu as G
from tests import test_gpu_linear as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_mod():
    if not G.have_gpu():
        pytest.skip("no HIP device")
    import torch
    from sparse_mixture_experts_20_amd import binding as B
    B.lib()
    return torch


def test_relu_gradient_where_z_is_nan(torch_mod):
    """The forward keeps a NaN in z; the backward passes its gradient on, as
    autograd's ReLU does, instead of 0."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    bf = torch.bfloat16
    N, K, M = 40, 16, 24
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    z = torch.randn((N, M), generator=g, device="cuda").to(bf)
    z[3, 5], z[3, 6], z[7, 0], z[9, 1] = float("nan"), 0.0, float("-inf"), float("inf")
    dout = torch.randn((N, M), generator=g, device="cuda").to(bf)
    x = torch.eye(N, K, device="cuda").to(bf)
    W = torch.eye(M, K, device="cuda").to(bf)
    dx, dW, db = B.linear_backward(x, W, z, dout, act="relu")
    zr = z.float().requires_grad_(True)
    want, = torch.autograd.grad(torch.relu(zr), zr, dout.float())
    assert float(want[3, 5]) == float(dout[3, 5]) != 0.0
    # one term per element: W and x are cut from the identity
    assert torch.equal(dx, want[:, :K])
    assert torch.equal(dW, want[:K].t())


def test_bias_gradient_of_the_widest_product(torch_mod):
    """M = 2^28 neurons, the most that is taken: sums of small whole numbers."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    bf = torch.bfloat16
    M = 1 << 28
    G.say(f"[linear backward] db of M={M}")
    x = torch.zeros((3, 8), dtype=bf, device="cuda")
    W = torch.empty((M, 8), dtype=bf, device="cuda")
    dout = torch.randint(-8, 9, (3, M), device="cuda", dtype=torch.int8).to(bf)
    _, _, db = B.linear_backward(x, W, None, dout, need_dx=False, need_dW=False)
    torch.cuda.synchronize()
    assert torch.equal(db, dout[0].float() + dout[1].float() + dout[2].float())


def _whole(torch, g, shape, most, dtype):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda",
                         dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("N,K,M,act,bias,residual", T.SHAPES)
def test_forward_of_whole_numbers(torch_mod, N, K, M, act, bias, residual):
    """out (ReLU or none) and z: the float64 result rounded once. Sums of
    magnitudes stay below 16 K < 2^24."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    bf = torch.bfloat16
    act = "none" if act == "none" else "relu"
    g = torch.Generator(device="cuda")
    g.manual_seed(N + K)
    x, W = _whole(torch, g, (N, K), 3, bf), _whole(torch, g, (M, K), 3, bf)
    b = _whole(torch, g, (M,), 100, torch.float32) if bias else None
    r = _whole(torch, g, (N, M), 100, bf) if residual else None
    G.say(f"[linear values] N={N} K={K} M={M} {act}")
    out, z = B.linear(x, W, b, act=act, residual=r, keep_z=True)
    torch.cuda.synchronize()
    want = x.double() @ W.double().t()
    if b is not None:
        want = want + b.double()
    assert torch.equal(z, want.to(bf))
    want = want.clamp(min=0) if act == "relu" else want
    assert torch.equal(out, (want if r is None else want + r.double()).to(bf))


@pytest.mark.parametrize("grads", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M,act", T.BACKWARD)
def test_backward_of_whole_numbers(torch_mod, N, K, M, act, grads):
    """dx, dW and db (ReLU or none): fp32 gradients exactly, bf16 ones rounded once."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    bf = torch.bfloat16
    dt = torch.float32 if grads == "f32" else bf
    act = "none" if act == "none" else "relu"
    g = torch.Generator(device="cuda")
    g.manual_seed(N + K)
    x, W = _whole(torch, g, (N, K), 3, bf), _whole(torch, g, (M, K), 3, bf)
    z = _whole(torch, g, (N, M), 3, bf) if act == "relu" else None
    dout = _whole(torch, g, (N, M), 3, bf)
    G.say(f"[linear values] backward N={N} K={K} M={M} {act} {grads}")
    dx, dW, db = B.linear_backward(x, W, z, dout, act=act, dx_dtype=dt, dW_dtype=dt)
    torch.cuda.synchronize()
    dz = dout.double() if z is None else dout.double() * (z > 0)
    assert torch.equal(dx, (dz @ W.double()).to(dt))
    assert torch.equal(dW, (dz.t().contiguous() @ x.double()).to(dt))
    assert torch.equal(db.double(), dz.sum(0))


def _norm_error(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("N,K,M,act,bias,residual", T.SHAPES)
def test_forward_distance_in_the_2_norm(torch_mod, N, K, M, act, bias, residual):
    """Each output is rounded once (2^-8 of it); its fp32 sum has at most 64
    dependent partial sums per range of 2048 columns, 2^-24 each, below 2^-12
    together at these lengths; the GELU formula adds 2.2e-7."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    x, W = T._randn(torch, (N, K), bf, 1), T._randn(torch, (M, K), bf, 2, K ** -0.5)
    b = T._randn(torch, (M,), torch.float32, 3, 0.5) if bias else None
    r = T._randn(torch, (N, M), bf, 4) if residual else None
    out, z = B.linear(x, W, b, act=act, residual=r, keep_z=True)
    y, z64, _, _ = P.linear(x, W, b, act, r)
    limit = 2.0 ** -8 + 2.0 ** -12
    errors = _norm_error(out, y), _norm_error(z, z64)
    G.say(f"[linear values] N={N} K={K} M={M} {act}: {errors[0]:.2e} {errors[1]:.2e}")
    assert max(errors) <= limit


@pytest.mark.parametrize("grads", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,M,act", T.BACKWARD)
def test_backward_distance_in_the_2_norm(torch_mod, N, K, M, act, grads):
    """dz is rounded once with an activation: a gradient is a sum of products
    with errors of at most 2^-8 of each, of independent signs, so its error in
    the 2-norm is that of the products: at most 2^-8 of sqrt(sum dz^2 W^2) over
    all, which is what the gradient of independent values of mean 0 measures
    (within a quarter at the smallest extents here, 8). A stored bf16 gradient
    is rounded once more. db sums fp32 values."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    dt = torch.float32 if grads == "f32" else bf
    x, W = T._randn(torch, (N, K), bf, 1), T._randn(torch, (M, K), bf, 2, K ** -0.5)
    z = T._randn(torch, (N, M), bf, 3) if act != "none" else None
    dout = T._randn(torch, (N, M), bf, 4)
    dx, dW, db = B.linear_backward(x, W, z, dout, act=act, dx_dtype=dt, dW_dtype=dt)
    ref = P.linear_backward(x, W, z, dout, act)
    limit = 2.0 ** -12
    limit += 1.25 * 2.0 ** -8 if act == "gelu" else 0.0
    limit += 2.0 ** -8 if grads == "bf16" else 0.0
    errors = _norm_error(dx, ref["dx"][0]), _norm_error(dW, ref["dW"][0])
    G.say(f"[linear values] backward N={N} K={K} M={M} {act} {grads}: "
          f"{errors[0]:.2e} {errors[1]:.2e} of {limit:.2e}")
    assert max(errors) <= limit
    assert _norm_error(db, ref["db"][0]) <= 2.0 ** -12
