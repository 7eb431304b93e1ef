"""moe_router_ex and moe_router_backward where an elementwise bound would not tell
a fault: bf16 gradients against the rounded float64 ones."""
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


@pytest.mark.parametrize("score,renorm,aux", [("softmax", False, False), ("softmax", True, True),
                                              ("sigmoid", False, True)])
def test_bf16_dx_of_all_scores(torch_mod, score, renorm, aux):
    """A bf16 dx of E values a token is the float64 one rounded, but for values next
    to the border of two steps. Products as accurate as fp32 ones leave a relative
    error of about 2^-22, so the border (every 2^-8 to 2^-7 of the value) is met by 2^-14
    to 2^-13 of the elements; with operands of 16 bits by 2^-10 to 2^-8. Limit: 2^-11."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain_route as R
    N, d, E, k = 512, 1024, 64, 4
    g = _gen(torch, 3)
    x = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((E, d), generator=g, device="cuda") / d ** 0.5
    idx, _, p = B.route(x, W, k, score=score, export_scores=True)
    dgate = torch.randn((N, k), generator=g, device="cuda")
    dp = torch.randn((N, E), generator=g, device="cuda") if aux else None
    dx, _ = B.route_backward(x, W, idx, p, dgate, dscores=dp, score=score, renormalize=renorm,
                             dx_dtype=torch.bfloat16)
    want = R.backward(x, W, idx, p, dgate, dp, None, score, renorm, 1.0)["dx"][0]
    off = float((dx != want.to(torch.bfloat16)).double().mean())
    G.say(f"[route backward] {score} renorm={renorm} aux={aux}: {off:.2e} of dx rounded otherwise")
    assert off <= 2.0 ** -11


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,E", [(7168, 256), (4096, 64)])
def test_no_tokens_of_many_experts(torch_mod, d, E, dtype):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, W = torch.empty((0, d), device="cuda", dtype=dt), torch.ones((E, d), device="cuda")
    idx, gate, p = B.route(x, W, 4, groups=8, keep_groups=2, export_scores=True)
    assert idx.shape == (0, 4) and gate.shape == (0, 4) and p.shape == (0, E)


def test_more_tokens_than_a_launch_holds(torch_mod):
    """64 threads a token pass a launch's 2^32 at 2^26 tokens: rows at both ends and on
    both sides of the parts' borders are those of calls of their own, dW_g the sum of
    the rows' terms (fp32: 2^-20 of the sum of magnitudes, ds's own roundings; sums of n
    random signs add about sqrt(n) 2^-24 of one term, far less)."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    N, d, E, k = (1 << 26) + 77, 8, 2, 1
    g = _gen(torch, 1)
    x = torch.randint(-3, 4, (N, d), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    W = torch.randint(-16, 17, (E, d), generator=g, device="cuda").float() / 16
    dgate = torch.randint(-2, 3, (N, k), generator=g, device="cuda", dtype=torch.int8).float()
    part = 1 << 25
    ends = [slice(0, 1000), slice(N - 999, N)] + [slice(i * part - 500, i * part + 500)
                                                  for i in (1, 2)]
    for score in ("sigmoid", "softmax"):      # k and E values a token
        G.say(f"[route] {N} tokens, {score}")
        idx, gate, p = B.route(x, W, k, score=score, export_scores=True)
        dx, dW = B.route_backward(x, W, idx, p, dgate, score=score)
        for s in ends:
            one = B.route(x[s], W, k, score=score, export_scores=True)
            assert all(torch.equal(a[s], b) for a, b in zip((idx, gate, p), one))
            alone, _ = B.route_backward(x[s], W, idx[s], p[s], dgate[s], score=score)
            assert torch.equal(dx[s], alone)
        want = torch.zeros((E, d), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for t in range(0, N, 1 << 23):
            q, i, xs = p[t:t + (1 << 23)].double(), idx[t:t + (1 << 23)].long(), x[t:t + (1 << 23)]
            up = torch.zeros_like(q).scatter_(1, i, dgate[t:t + (1 << 23)].double())
            ds = q * (1 - q) * up if score == "sigmoid" else q * (up - (q * up).sum(1, keepdim=True))
            for e in range(E):    # (a product of so many rows is slow in float64)
                terms = ds[:, e:e + 1] * xs.double()
                want[e] += terms.sum(0)
                size[e] += terms.abs().sum(0)
        assert bool(((dW.double() - want).abs() <= 2.0 ** -20 * size).all())
        del idx, gate, p, dx
