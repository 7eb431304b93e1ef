"""moe_linear and moe_linear_backward at values where a check of magnitudes
would not tell a fault: NaN, and the largest extents."""
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
