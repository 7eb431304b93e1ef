"""A launch of 2^32 threads or more is refused: HIP would run the low 32 bits of them and
leave the rest of the rows as they were."""
import pytest

from tests import _gpu as G

pytestmark = pytest.mark.gpu


def test_router_past_a_launch():
    if not G.have_gpu():
        pytest.skip("no HIP device")
    import torch
    from sparse_mixture_experts_20_amd import binding as B
    N = (1 << 26) + 64          # 64 threads a token
    x = torch.zeros((N, 1), device="cuda")
    W = torch.zeros((2, 1), device="cuda")
    with pytest.raises(B.MoeError) as e:
        B.router(x, W, None, 1)
    assert e.value.code == -8
    # the library goes on, and the last row of the largest launch is written (workgroups
    # of 4 tokens and 256 threads: 2^26 - 4 tokens are 2^32 - 256 threads, one more is 2^32)
    n = (1 << 26) - 4
    idx, gate = B.router(x[:n], W, None, 1)
    assert bool((gate == 1).all()) and not bool(idx.any())
