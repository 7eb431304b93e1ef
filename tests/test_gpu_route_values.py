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


@pytest.mark.parametrize("aux", [False, True])
@pytest.mark.parametrize("low", [(-200.0, -201.0), (-95.0, -96.5), (-88.5, -87.0), (0.5, 0.25)])
def test_gradient_of_gates_whose_scores_underflow(torch_mod, low, aux):
    """Renormalised softmax gates of experts that a bias forces: the gradient is that of
    the gates the forward wrote (float64 autograd from the logits), which its scores no
    longer hold: p is 0, or below 2^-126 with 10 to 22 bits. Bound: 20 roundings of
    2^-24 of the operands' sizes, as few as ds takes."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    N, d, E, k, scale = 6, 8, 4, 2, 2.5
    g = _gen(torch, 8)
    x = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.zeros((E, d), device="cuda")
    W[:, 0] = torch.tensor([0.0, 0.5, -0.25, 0.0], device="cuda")
    x[:, 0] = 0.0                       # (the logits are the noise, dx sees W_g)
    noise = torch.tensor([[0.0, *low, -300.0]] * N, device="cuda")
    bias = torch.tensor([0.0, 3.0, 2.0, 0.0], device="cuda")
    rule = dict(score="softmax", renormalize=True, scale=scale)
    idx, gate, p = B.route(x, W, k, noise=noise, bias=bias, export_scores=True, **rule)
    assert bool(((idx == 1) | (idx == 2)).all())
    dgate = torch.randn((N, k), generator=g, device="cuda")
    dp = torch.randn((N, E), generator=g, device="cuda") if aux else None
    dx, dW = B.route_backward(x, W, idx, p, dgate, dscores=dp, gate=gate, **rule)
    s = noise.double().requires_grad_()
    loss = (scale * torch.softmax(s.gather(1, idx.long()), 1) * dgate.double()).sum()
    if aux:
        loss = loss + (torch.softmax(s, 1) * dp.double()).sum()
    ds, = torch.autograd.grad(loss, s)
    size = 2 * scale * float(dgate.abs().max()) + (2 * float(dp.abs().max()) if aux else 0.0)
    tol = 20 * 2.0 ** -24 * size
    assert bool(((dW.double() - ds.t() @ x.double()).abs()
                 <= tol * x.double().abs().sum(0)).all())
    assert bool(((dx.double() - ds @ W.double()).abs() <= tol * W.double().abs().sum(0)).all())


def test_gates_given_to_the_backward(torch_mod):
    """Where nothing underflows the gates' shares are the scores' to a few fp32 steps,
    for both scores; gates that are not renormalised are not read."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    N, d, E, k = 333, 264, 40, 6
    g = _gen(torch, 9)
    x = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((E, d), generator=g, device="cuda") / d ** 0.5
    dgate = torch.randn((N, k), generator=g, device="cuda")
    for score in ("softmax", "sigmoid"):
        rule = dict(score=score, renormalize=True, scale=0.75)
        idx, gate, p = B.route(x, W, k, export_scores=True, **rule)
        idx[5, 2], idx[6] = -1, E             # no experts: their gates are not read
        gate[5, 2], gate[6] = float("nan"), float("nan")
        a = B.route_backward(x, W, idx, p, dgate, gate=gate, **rule)
        rows = torch.ones(N, dtype=torch.bool, device="cuda")
        rows[5] = False                       # (its shares are of the gates that are left)
        b = B.route_backward(x, W, idx, p, dgate, **rule)
        assert float((a[0] - b[0])[rows].norm()) <= 2.0 ** -20 * float(b[0].norm())
        assert bool(torch.isfinite(a[0]).all()) and bool(torch.isfinite(a[1]).all())
        rule["renormalize"] = False
        a = B.route_backward(x, W, idx, p, dgate, gate=gate, **rule)
        b = B.route_backward(x, W, idx, p, dgate, **rule)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_expert_takes_nothing_of_the_weights(torch_mod):
    """A token whose ids are outside [0, E) has dx = dres, also where rows of W_g are not
    finite (with k values a token no other expert's row is read)."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    N, d, E, k = 40, 264, 6, 3
    g = _gen(torch, 2)
    x = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((E, d), generator=g, device="cuda") / d ** 0.5
    idx, _, p = B.route(x, W, k, score="sigmoid", export_scores=True)
    idx = torch.where(idx == 0, torch.full_like(idx, E), idx)
    idx[3] = torch.tensor([-1, E, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    dgate = torch.randn((N, k), generator=g, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        dres = torch.randn((N, d), generator=g, device="cuda").to(dt)
        kw = dict(dres=dres, score="sigmoid", need_dW=False, dx_dtype=dt)
        want, _ = B.route_backward(x, W, idx, p, dgate, **kw)
        V = W.clone()
        V[0, ::2], V[0, 1::2] = float("inf"), float("nan")
        got, _ = B.route_backward(x, V, idx, p, dgate, **kw)
        assert torch.equal(got, want) and torch.equal(got[3], dres[3])
