"""moe_layer_norm and moe_layer_norm_backward against their float64 forms:
both types, widths on both sides of every variant (waves, workgroups, the
widest row), odd widths, one row to more rows than the grid walks at once."""
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


# (N, d) for bf16 and fp32: the narrowest and widest row of each variant, odd rows
BF16 = [(1, 8), (5, 512), (3, 520), (700, 1024), (2, 1032), (513, 4096), (4, 4104), (33, 8192),
        (3, 8200), (7, 16384), (9001, 64), (2500, 768)]
F32 = [(1, 1), (1, 4), (4, 3), (6, 255), (3, 257), (5, 512), (2, 516), (2049, 1023), (3, 1025),
       (3, 2052), (2, 4097), (3, 4100), (5, 8196), (2, 16383), (3, 16384), (9001, 12)]


def _rows(torch, N, d, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.randn((N, d), generator=g, device="cuda") * scale + shift
    return t.to(dtype)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype,N,d", [("bf16", *s) for s in BF16] + [("f32", *s) for s in F32])
def test_forward_and_backward(torch_mod, dtype, N, d, residual):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    G.say(f"[norm] {dtype} N={N} d={d} residual={residual}")
    x = _rows(torch, N, d, dt, 1, 1.5, 0.75)
    r = _rows(torch, N, d, dt, 2) if residual else None
    w = 1.0 + 0.25 * _rows(torch, 1, d, torch.float32, 3)[0]
    b = _rows(torch, 1, d, torch.float32, 4)[0] if d % 3 else None
    out, h, mean, rstd = B.layer_norm(x, w, b, eps=1e-5, residual=r, stats=True)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(h, (x.float() + r.float()).to(dt))
    else:
        assert h is x
    y, m, rs, ey, em, er = P.layer_norm(h, w, b, 1e-5)
    P.close(out, y, P.stored(y, ey, dt), "out")
    P.close(mean, m, P.stored(m, em, torch.float32), "mean")
    P.close(rstd, rs, P.stored(rs, er, torch.float32), "rstd")
    dout = _rows(torch, N, d, dt, 5)
    dres = _rows(torch, N, d, dt, 6) if residual else None
    dx, dw, db = B.layer_norm_backward(h, w, mean, rstd, dout, dres=dres, bias=b is not None)
    torch.cuda.synchronize()
    ref = P.layer_norm_backward(h, w, mean, rstd, dout, dres)
    P.close(dx, ref["dx"][0], P.stored(*ref["dx"], dt), "dx")
    P.close(dw, ref["dw"][0], P.stored(*ref["dw"], torch.float32), "dw")
    assert (db is None) == (b is None)
    if db is not None:
        P.close(db, ref["db"][0], P.stored(*ref["db"], torch.float32), "db")
    # the same call again gives the same bits
    again = B.layer_norm_backward(h, w, mean, rstd, dout, dres=dres, bias=b is not None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_large_mean_and_special_rows(torch_mod):
    """A mean 1000 times the spread, a constant row, and rows holding an
    infinity or a NaN, which stay theirs."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    for d in (96, 3000, 9000):
        x = _rows(torch, 6, d, torch.float32, 7, 1.0, 1000.0)
        x[1] = 2.5
        x[3, 5] = float("inf")
        x[4, d - 1] = float("nan")
        w, b = torch.full((d,), 1.5, device="cuda"), torch.full((d,), 0.5, device="cuda")
        out, _, mean, rstd = B.layer_norm(x, w, b, stats=True)
        ok = torch.tensor([0, 1, 2, 5], device="cuda")
        y, m, rs, ey, em, er = P.layer_norm(x[ok], w, b, 1e-5)
        P.close(out[ok], y, P.stored(y, ey, torch.float32), "out")
        assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(out[4]).all())


def test_buffers_may_be_reused(torch_mod):
    """h over x, out over the residual; dx over dout: the same bits as apart."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    for N, d in ((3000, 768), (600, 7168)):
        x, r = _rows(torch, N, d, torch.bfloat16, 1), _rows(torch, N, d, torch.bfloat16, 2)
        w = 1.0 + 0.25 * _rows(torch, 1, d, torch.float32, 3)[0]
        out, h, mean, rstd = B.layer_norm(x, w, residual=r, stats=True)
        x2, r2 = x.clone(), r.clone()
        B.layer_norm(x2, w, residual=r2, h=x2, out=r2)
        assert torch.equal(x2, h) and torch.equal(r2, out)
        g, gr = _rows(torch, N, d, torch.bfloat16, 4), _rows(torch, N, d, torch.bfloat16, 5)
        dx, dw, db = B.layer_norm_backward(h, w, mean, rstd, g, dres=gr)
        for buf in (0, 1):
            g2, gr2 = g.clone(), gr.clone()
            got = B.layer_norm_backward(h, w, mean, rstd, g2, dres=gr2, dx=(g2, gr2)[buf])
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


def test_no_rows(torch_mod):
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    x = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    out, _, mean, rstd = B.layer_norm(x, w, w, stats=True)
    dx, dw, db = B.layer_norm_backward(x, w, mean, rstd, x)
    assert out.shape == (0, 64) and dx.shape == (0, 64)
    assert not bool(dw.any()) and not bool(db.any())


def test_gradient_against_differences(torch_mod):
    """Central differences of the kernel's own fp32 forward along random
    directions: the forward is exact to about 1e-6 of values of order one, so
    with a step of 2^-6 the quotient of a sum of 24 x 40 such terms holds to
    about 1e-6 * sqrt(960) / 2^-6 + third-order terms (2^-12): 2e-3 of the
    gradient's norm."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    N, d = 24, 40
    x = _rows(torch, N, d, torch.float32, 1)
    w, b = 1.0 + 0.25 * _rows(torch, 1, d, torch.float32, 2)[0], _rows(torch, 1, d, torch.float32, 3)[0]
    c = _rows(torch, N, d, torch.float32, 4)
    loss = lambda x, w, b: float((B.layer_norm(x, w, b)[0].double() * c.double()).sum())  # noqa: E731
    _, _, mean, rstd = B.layer_norm(x, w, b, stats=True)
    grads = B.layer_norm_backward(x, w, mean, rstd, c)
    h = 2.0 ** -6
    for seed in range(3):
        for i, p in enumerate((x, w, b)):
            v = _rows(torch, 1, p.numel(), torch.float32, 10 + seed).reshape(p.shape)
            args = [x, w, b]
            args[i] = p + h * v
            hi = loss(*args)
            args[i] = p - h * v
            lo = loss(*args)
            want = (hi - lo) / (2 * h)
            got = float((grads[i].double() * v.double()).sum())
            scale = float(grads[i].double().norm()) * float(v.double().norm())
            assert abs(got - want) <= 2e-3 * scale, (i, got, want)


def test_offsets_past_32_bits(torch_mod):
    """More than 2^31 elements: the first and last rows, and column sums of a
    dout that is zero but for some of those rows."""
    torch = torch_mod
    from sparse_mixture_experts_20_amd import binding as B
    from tests import _plain as P
    bf = torch.bfloat16
    N, d = 300007, 7168
    rows = torch.tensor([0, 5, 150001, N - 3, N - 1], device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.empty((N, d), dtype=bf, device="cuda").normal_(generator=g)
    r = torch.empty((N, d), dtype=bf, device="cuda").normal_(generator=g)
    w, b = 1.0 + 0.25 * _rows(torch, 1, d, torch.float32, 3)[0], _rows(torch, 1, d, torch.float32, 4)[0]
    out, h, mean, rstd = B.layer_norm(x, w, b, residual=r, stats=True)
    torch.cuda.synchronize()
    assert torch.equal(h[rows], x[rows] + r[rows])
    y, m64, r64, ey, em, er = P.layer_norm(h[rows], w, b, 1e-5)
    P.close(out[rows], y, P.stored(y, ey, bf), "out")
    P.close(mean[rows], m64, em + 2.0 ** -24 * m64.abs(), "mean")
    dout = out.zero_()
    dout[rows] = _rows(torch, len(rows), d, bf, 5)
    G.say("[norm] past 32 bits: backward")
    dx, dw, db = B.layer_norm_backward(h, w, mean, rstd, dout)
    torch.cuda.synchronize()
    ref = P.layer_norm_backward(h[rows], w, mean[rows], rstd[rows], dout[rows], None)
    P.close(dx[rows], ref["dx"][0], P.stored(*ref["dx"], bf), "dx")
    P.close(dw, ref["dw"][0], P.stored(*ref["dw"], torch.float32), "dw")
    P.close(db, ref["db"][0], P.stored(*ref["db"], torch.float32), "db")
    dx[rows] = 0
    assert not bool(dx.any())
