"""moe_layer_norm and its backward with several rows for each workgroup of the
widest variants (1024 threads a row): their second and later rows, the column
sums carried over rows, and buffers used in place there."""
import pytest

from tests import _gpu as G
from tests import test_gpu_norm as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_mod():
    if not G.have_gpu():
        pytest.skip("no HIP device")
    import torch
    from sparse_mixture_experts_20_amd import binding as B
    B.lib()
    return torch


# more rows than the 512 (forward) and 256 (backward) workgroups of these variants
ROWS = [("bf16", 1100, 8200), ("bf16", 700, 16384), ("f32", 1100, 4100), ("f32", 700, 16384),
        ("f32", 1100, 1025), ("f32", 700, 4097), ("f32", 600, 16383), ("f32", 1100, 8196)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype,N,d", ROWS)
def test_many_wide_rows(torch_mod, dtype, N, d, residual):
    T.test_forward_and_backward(torch_mod, dtype, N, d, residual)


@pytest.mark.parametrize("dtype,N,d", ROWS)
def test_buffers_reused_by_wide_rows(torch_mod, dtype, N, d):
    """h over x and out over the residual; dx over dout or dres: the bits of
    separate buffers, in every row."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    G.say(f"[norm] in place, {dtype} N={N} d={d}")
    x, r = T._rows(torch, N, d, dt, 1), T._rows(torch, N, d, dt, 2)
    w = 1.0 + 0.25 * T._rows(torch, 1, d, torch.float32, 3)[0]
    out, h, mean, rstd = B.layer_norm(x, w, residual=r, stats=True)
    x2, r2 = x.clone(), r.clone()
    B.layer_norm(x2, w, residual=r2, h=x2, out=r2)
    assert torch.equal(x2, h) and torch.equal(r2, out)
    x2, r2 = x.clone(), r.clone()
    B.layer_norm(x2, w, residual=r2, h=r2, out=x2)
    assert torch.equal(r2, h) and torch.equal(x2, out)
    g, gr = T._rows(torch, N, d, dt, 4), T._rows(torch, N, d, dt, 5)
    dx, dw, db = B.layer_norm_backward(h, w, mean, rstd, g, dres=gr)
    for buf in (0, 1):
        g2, gr2 = g.clone(), gr.clone()
        got = B.layer_norm_backward(h, w, mean, rstd, g2, dres=gr2, dx=(g2, gr2)[buf])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
