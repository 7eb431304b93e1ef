"""The operators around the sparse MoE layer that complete a transformer's
feed-forward half, each as a measurable case: the whole MoE layer for a few
tokens, the linear product with bias, activation and residual (and its
backward), and the layer norm (and its backward).

With ``own`` false ``run`` computes an operator in its plain form (elementary
torch operations in fp32, rounded once at the end); with ``own`` true it makes
the calls a user makes of this package. ``exact`` computes the same outputs
from the operators' definitions in float64.

Shapes: "nanomoe", "mixtral" and "finegrained" are this repository's layer
shapes (d = 768 / 4096 / 7168, d_ff = 3072 / 14336 / 2048, E = 8 / 8 / 256,
k = 2 / 2 / 8).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # decoding one sequence through the nanoMoE layer of the slides (GELU,
        # biases): the smallest call, all latency
        dict(name="few_token_nanomoe", op="few", N=1, d=768, E=8, k=2, d_ff=3072, cf=1.25,
             dtype="bf16", act="gelu", bias=True, sigma=1.0),
        # decoding one sequence through the Mixtral-shaped layer: two experts'
        # weights stream from HBM
        dict(name="few_token_mixtral", op="few", N=1, d=4096, E=8, k=2, d_ff=14336, cf=1.25,
             dtype="bf16", act="relu", bias=False, sigma=0.0),
        # a decode batch (odd, near the largest) through the fine-grained
        # layer: most of its 256 experts are hit by one to six tokens each
        dict(name="few_batch_finegrained", op="few", N=61, d=7168, E=256, k=8, d_ff=2048, cf=1.5,
             dtype="bf16", act="relu", bias=False, sigma=0.0),
        # a small fp32 layer of odd widths, some assignments past the capacity
        dict(name="few_f32_odd", op="few", N=21, d=515, E=6, k=3, d_ff=1021, cf=1.0,
             dtype="f32", act="gelu", bias=True, sigma=0.5),
        # shared expert's up-projection for a few decoded tokens (GELU, bias)
        dict(name="linear_decode", op="linear", N=4, K=7168, M=2048, act="gelu", bias=True,
             residual=False, z=False),
        # shared expert's down-projection over a prefill batch, added to the
        # routed experts' output
        dict(name="linear_residual", op="linear", N=8192, K=2048, M=7168, act="none", bias=True,
             residual=True, z=False),
        # backward of a dense feed-forward layer's up-projection (GELU)
        dict(name="linear_bwd_gelu", op="linear_bwd", N=4096, K=4096, M=14336, act="gelu",
             bias=True, grads="bf16"),
        # backward of a small dense layer's projection over a ragged batch,
        # fp32 weight gradient
        dict(name="linear_bwd_ragged", op="linear_bwd", N=2047, K=3072, M=768, act="none",
             bias=True, grads="f32"),
        # pre-norm of a prefill batch: residual add, norm, statistics kept
        dict(name="norm_prefill", op="norm", N=8192, d=7168, dtype="bf16", bias=True,
             residual=True),
        # pre-norm of one decoded token
        dict(name="norm_token", op="norm", N=1, d=4096, dtype="bf16", bias=True, residual=True),
        # its backward over the same batch, with the residual path's gradient
        dict(name="norm_bwd", op="norm_bwd", N=8192, d=7168, dtype="bf16", bias=True,
             residual=True),
        # a ragged fp32 batch of odd width
        dict(name="norm_bwd_f32_odd", op="norm_bwd", N=2049, d=1023, dtype="f32", bias=True,
             residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult8(v):
    return max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["few", "few", "few", "linear", "linear", "linear_bwd", "norm", "norm_bwd"])
    if op == "few":
        f32 = rng.random() < 0.2
        E = _log(rng, 2, 256)
        k = min(E, rng.choice([1, 2, 2, 3, 4, 6, 8]))
        N = rng.choice([1, rng.randint(1, 16), rng.randint(1, 64)])
        d, d_ff = _log(rng, 64, 1100 if f32 else 7168), _log(rng, 64, 1100 if f32 else 14336)
        if not f32:
            d, d_ff = _mult8(d), _mult8(d_ff)
            while E * d * d_ff > 256 * 7168 * 2048:
                E = max(k, E // 2)
                d_ff = _mult8(d_ff * 3 // 4)
        return dict(op=op, N=N, d=d, E=E, k=k, d_ff=d_ff, cf=rng.choice([0.75, 1.0, 1.25, 1.5]),
                    dtype="f32" if f32 else "bf16", act=rng.choice(["relu", "gelu"]),
                    bias=rng.random() < 0.5, sigma=rng.choice([0.0, 0.5]))
    if op in ("linear", "linear_bwd"):
        N = rng.choice([rng.randint(1, 64), _log(rng, 1, 8192), _log(rng, 64, 8192)])
        K, M = _mult8(_log(rng, 64, 8192)), _mult8(_log(rng, 64, 8192))
        most = 8192 * 2048 * 7168
        while N * K * M > most:
            N = max(1, N // 2)
        act = rng.choice(["none", "relu", "gelu"])
        if op == "linear":
            return dict(op=op, N=N, K=K, M=M, act=act, bias=rng.random() < 0.7,
                        residual=rng.random() < 0.5, z=rng.random() < 0.5)
        return dict(op=op, N=N, K=K, M=M, act=act, bias=rng.random() < 0.7,
                    grads="f32" if act == "none" and rng.random() < 0.5 else "bf16")
    f32 = rng.random() < 0.4
    d = _log(rng, 16, 12288)
    if not f32:
        d = _mult8(d)
    N = _log(rng, 1, 16384)
    while N * d * (2 if f32 else 1) > 8192 * 7168:
        N = max(1, N // 2)
    return dict(op=op, N=N, d=d, dtype="f32" if f32 else "bf16", bias=rng.random() < 0.7,
                residual=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, shape, dtype, std=1.0, mean=0.0):
    t = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    if std != 1.0:
        t.mul_(std)
    if mean != 0.0:
        t.add_(mean)
    return t


def _inputs(case, seed):
    """The case's input tensors, from the seed alone (the same for every caller)."""
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 1000003 + 17)
    s = dict(case)
    f32 = torch.float32
    if case["op"] == "few":
        N, d, E, k, d_ff = (case[n] for n in ("N", "d", "E", "k", "d_ff"))
        dt = DTYPES[case["dtype"]]
        s["W_up"] = _randn(g, (E, d_ff, d), dt, 1.0 / math.sqrt(d))
        s["W_down"] = _randn(g, (E, d, d_ff), dt, 1.0 / math.sqrt(d_ff))
        s["W_g"] = _randn(g, (E, d), f32, 1.0 / math.sqrt(d))
        s["b_up"] = _randn(g, (E, d_ff), f32, 0.1) if case["bias"] else None
        s["b_down"] = _randn(g, (E, d), f32, 0.1) if case["bias"] else None
        s["noise"] = _randn(g, (N, E), f32, case["sigma"]) if case["sigma"] else None
        # Rows whose ranking is ambiguous in fp32 (two of the top k + 1 scores
        # nearer than 1e-4) are drawn again: ids and slots are whole numbers.
        x = _randn(g, (N, d), dt)
        m = min(k + 1, E)
        for _ in range(200):
            sc = x.double() @ s["W_g"].double().t()
            if s["noise"] is not None:
                sc = sc + s["noise"].double()
            top = sc.topk(m, dim=1).values
            near = ((top[:, :-1] - top[:, 1:]) < 1e-4).any(dim=1) if m > 1 else None
            if near is None or not bool(near.any()):
                break
            x = torch.where(near[:, None], _randn(g, (N, d), dt), x)
        s["x"] = x
    elif case["op"] in ("linear", "linear_bwd"):
        N, K, M = case["N"], case["K"], case["M"]
        bf = torch.bfloat16
        s["x"] = _randn(g, (N, K), bf)
        s["W"] = _randn(g, (M, K), bf, 1.0 / math.sqrt(K))
        if case["op"] == "linear":
            s["b"] = _randn(g, (M,), f32, 0.1) if case["bias"] else None
            s["r"] = _randn(g, (N, M), bf) if case["residual"] else None
        else:
            s["z"] = _randn(g, (N, M), bf) if case["act"] != "none" else None
            s["dout"] = _randn(g, (N, M), bf)
    else:
        N, d = case["N"], case["d"]
        dt = DTYPES[case["dtype"]]
        # rows of a residual stream: a mean and a scale of their own
        scale = torch.exp(_randn(g, (N, 1), f32, 0.5))
        shift = _randn(g, (N, 1), f32, 0.5)
        s["x"] = (_randn(g, (N, d), f32) * scale + shift).to(dt)
        s["w"] = _randn(g, (d,), f32, 0.2, 1.0)
        s["b"] = _randn(g, (d,), f32, 0.2) if case["bias"] else None
        s["r"] = _randn(g, (N, d), dt) if case["residual"] else None
        if case["op"] == "norm_bwd":
            s["dout"] = _randn(g, (N, d), dt)
            x64 = s["x"].double()
            mean = x64.mean(dim=1)
            s["mean"] = mean.float()
            s["rstd"] = (1.0 / torch.sqrt(((x64 - mean[:, None]) ** 2).mean(dim=1) + EPS)).float()
    return s


EPS = 1e-5


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # what a program keeps beside its tensors: the layer's handle (weight
        # descriptors, workspace, output and routing buffers), the scratch of a call
        from sparse_mixture_experts_20_amd import binding as B
        if case["op"] == "few":
            s["layer"] = B.FewLayer(s["W_g"], s["W_up"], s["W_down"], case["k"], case["cf"],
                                    act=case["act"], b_up=s["b_up"], b_down=s["b_down"],
                                    max_tokens=case["N"], export=True)
        elif case["op"] == "linear":
            n = B.linear_workspace_size(case["N"], case["K"], case["M"])
            s["ws"] = B.alloc_workspace(n) if n else None
        elif case["op"] == "linear_bwd":
            n = B.linear_backward_workspace_size(case["N"], case["K"], case["M"], case["act"])
            s["ws"] = B.alloc_workspace(n) if n else None
        elif case["op"] == "norm_bwd":
            n = B.layer_norm_backward_workspace_size(case["N"], case["d"])
            s["ws"] = B.alloc_workspace(n) if n else None
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(
        2 * math.pi)


def _route(scores, k, E, cf):
    """ids, gates and capacity slots (-1: dropped) of the scores [N, E]."""
    N = scores.shape[0]
    top, idx = torch.sort(scores, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    ex = torch.exp(top - top[:, :1])
    gate = ex / ex.sum(dim=1, keepdim=True)
    # rank of each assignment among its expert's, first choices of every token first
    flat = idx.t().reshape(-1)
    hot = (flat[:, None] == torch.arange(E, device=idx.device)).to(torch.int64)
    rank = (hot.cumsum(0) - 1).gather(1, flat[:, None])[:, 0].reshape(k, N).t()
    cap = math.ceil(cf * (k * N) / E)
    return idx, gate, torch.where(rank < cap, rank, torch.full_like(rank, -1))


def _plain_few(s):
    N, d, E, k, d_ff = (s[n] for n in ("N", "d", "E", "k", "d_ff"))
    x = s["x"].float()
    scores = x @ s["W_g"].t()
    if s["noise"] is not None:
        scores = scores + s["noise"]
    idx, gate, slot = _route(scores, k, E, s["cf"])
    if N * k < E:   # the chosen experts' weights, one copy an assignment
        a = idx.reshape(-1)
        z = torch.bmm(s["W_up"][a].float(), x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        if s["b_up"] is not None:
            z = z + s["b_up"][a]
        y = torch.bmm(s["W_down"][a].float(), _act(z, s["act"])[:, :, None])[:, :, 0]
        if s["b_down"] is not None:
            y = y + s["b_down"][a]
        y = y.reshape(N, k, d)
    else:           # every expert for every token, then each token's choices
        z = (x @ s["W_up"].float().reshape(E * d_ff, d).t()).reshape(N, E, d_ff)
        if s["b_up"] is not None:
            z = z + s["b_up"]
        h = _act(z, s["act"]).permute(1, 0, 2).contiguous()
        y = torch.bmm(h, s["W_down"].float().transpose(1, 2).contiguous())
        if s["b_down"] is not None:
            y = y + s["b_down"][:, None, :]
        y = y[idx, torch.arange(N, device=idx.device)[:, None]]
    out = torch.where((slot >= 0)[:, :, None], gate[:, :, None] * y, torch.zeros_like(y)).sum(1)
    return {"out": out.to(s["x"].dtype), "idx": idx.int(), "gate": gate, "slot": slot.int()}


def _plain_linear(s):
    z = s["x"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    out = _act(z, s["act"])
    if s["r"] is not None:
        out = out + s["r"].float()
    got = {"out": out.to(torch.bfloat16)}
    if s["z"]:
        got["z"] = z.to(torch.bfloat16)
    return got


def _plain_linear_bwd(s):
    dz = s["dout"].float()
    if s["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), s["act"])
    got = {"dx": (dz @ s["W"].float()).to(torch.bfloat16),
           "dW": (dz.t() @ s["x"].float()).to(DTYPES[s["grads"]])}
    if s["bias"]:
        got["db"] = dz.sum(dim=0)
    return got


def _plain_norm(s):
    h = s["x"]
    if s["r"] is not None:   # the residual stream, as it is kept
        h = (h.float() + s["r"].float()).to(h.dtype)
    v = h.float()
    mean = v.mean(dim=1)
    c = v - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1) + EPS)
    y = c * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    got = {"out": y.to(h.dtype), "mean": mean, "rstd": rstd}
    if s["r"] is not None:
        got["h"] = h
    return got


def _plain_norm_bwd(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dout"].float()
    gw = dy * s["w"]
    dx = s["rstd"][:, None] * (gw - gw.mean(dim=1, keepdim=True)
                               - xh * (gw * xh).mean(dim=1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    got = {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(dim=0)}
    if s["bias"]:
        got["db"] = dy.sum(dim=0)
    return got


PLAIN = {"few": _plain_few, "linear": _plain_linear, "linear_bwd": _plain_linear_bwd,
         "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


def _own(s):
    """The calls a user makes of this package."""
    from sparse_mixture_experts_20_amd import binding as B
    op = s["op"]
    if op == "few":
        out, st = s["layer"](s["x"], s["noise"])
        return {"out": out, "idx": st.idx, "gate": st.gate, "slot": st.slot}
    if op == "linear":
        out, z = B.linear(s["x"], s["W"], s["b"], act=s["act"], residual=s["r"],
                          keep_z=s["z"], workspace=s["ws"])
        return {"out": out, "z": z} if s["z"] else {"out": out}
    if op == "linear_bwd":
        dx, dW, db = B.linear_backward(s["x"], s["W"], s["z"], s["dout"], act=s["act"],
                                       bias=s["bias"], dx_dtype=torch.bfloat16,
                                       dW_dtype=DTYPES[s["grads"]], workspace=s["ws"])
        return {"dx": dx, "dW": dW, "db": db} if s["bias"] else {"dx": dx, "dW": dW}
    if op == "norm":
        out, h, mean, rstd = B.layer_norm(s["x"], s["w"], s["b"], eps=EPS, residual=s["r"],
                                          stats=True)
        got = {"out": out, "mean": mean, "rstd": rstd}
        if s["r"] is not None:
            got["h"] = h
        return got
    dx, dw, db = B.layer_norm_backward(s["x"], s["w"], s["mean"], s["rstd"], s["dout"],
                                       dres=s["r"], bias=s["bias"], workspace=s["ws"])
    return {"dx": dx, "dw": dw, "db": db} if s["bias"] else {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "few":
        N, d, E, k, d_ff = (case[n] for n in ("N", "d", "E", "k", "d_ff"))
        es = 4 if case["dtype"] == "f32" else 2
        hit = E * (1.0 - (1.0 - k / E) ** N)   # experts that at least one token takes
        return {"bytes": hit * 2 * d * d_ff * es + E * d * 4 + 2 * N * d * es
                + (hit * (d + d_ff) * 4 if case["bias"] else 0)
                + (N * E * 4 if case["sigma"] else 0) + N * k * 12,
                "flops": 4.0 * N * k * d * d_ff + 2.0 * N * E * d}
    if op == "linear":
        N, K, M = case["N"], case["K"], case["M"]
        return {"bytes": 2 * (N * K + M * K + N * M * (1 + case["residual"] + case["z"]))
                + (4 * M if case["bias"] else 0), "flops": 2.0 * N * K * M}
    if op == "linear_bwd":
        N, K, M = case["N"], case["K"], case["M"]
        gw = 4 if case["grads"] == "f32" else 2
        return {"bytes": 2 * (2 * N * K + M * K + N * M * (1 if case["act"] == "none" else 2))
                + gw * M * K + (4 * M if case["bias"] else 0), "flops": 4.0 * N * K * M}
    N, d = case["N"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        return {"bytes": N * d * es * (4 if case["residual"] else 2) + 8 * N
                + 4 * d * (1 + case["bias"]), "flops": 8.0 * N * d}
    return {"bytes": N * d * es * (4 if case["residual"] else 3) + 8 * N
            + 4 * d * (2 + case["bias"]), "flops": 14.0 * N * d}


# --------------------------------------------------------------------------
# the definitions in float64
# --------------------------------------------------------------------------
def _phi(z):
    """The standard normal distribution function."""
    return 0.5 * (1.0 + torch.erf(z / math.sqrt(2.0)))


def _exact_few(s):
    N, d, E, k = (s[n] for n in ("N", "d", "E", "k"))
    x, noise = s["x"].double(), s["noise"]
    score = x @ s["W_g"].double().t() + (0.0 if noise is None else noise.double())
    score = score.cpu()
    cap = math.ceil(s["cf"] * (k * N) / E)
    idx = torch.zeros((N, k), dtype=torch.int32)
    gate = torch.zeros((N, k), dtype=torch.float64)
    slot = torch.full((N, k), -1, dtype=torch.int32)
    for t in range(N):
        order = sorted(range(E), key=lambda e: (-float(score[t, e]), e))[:k]
        idx[t] = torch.tensor(order, dtype=torch.int32)
        gate[t] = torch.softmax(score[t, order], dim=0)
    rows = {e: [] for e in range(E)}
    for j in range(k):
        for t in range(N):
            e = int(idx[t, j])
            if len(rows[e]) < cap:
                slot[t, j] = len(rows[e])
                rows[e].append((t, j))
    out = torch.zeros((N, d), dtype=torch.float64, device=DEVICE)
    for e, members in rows.items():
        if not members:
            continue
        ts = torch.tensor([t for t, _ in members], device=DEVICE)
        gs = torch.tensor([float(gate[t, j]) for t, j in members], dtype=torch.float64,
                          device=DEVICE)
        z = x[ts] @ s["W_up"][e].double().t()
        if s["b_up"] is not None:
            z = z + s["b_up"][e].double()
        h = torch.relu(z) if s["act"] == "relu" else z * _phi(z)
        y = h @ s["W_down"][e].double().t()
        if s["b_down"] is not None:
            y = y + s["b_down"][e].double()
        out.index_add_(0, ts, gs[:, None] * y)
    return {"out": out, "idx": idx, "gate": gate, "slot": slot}


def _exact_linear(s):
    z = torch.mm(s["x"].double(), s["W"].double().t().contiguous())
    if s["b"] is not None:
        z += s["b"].double()
    out = {"none": lambda v: v, "relu": torch.relu, "gelu": lambda v: v * _phi(v)}[s["act"]](z)
    if s["r"] is not None:
        out = out + s["r"].double()
    return {"out": out, "z": z} if s["z"] else {"out": out}


def _exact_linear_bwd(s):
    dz = s["dout"].double()
    if s["act"] == "relu":
        dz = torch.where(s["z"] > 0, dz, torch.zeros_like(dz))
    elif s["act"] == "gelu":
        z = s["z"].double()
        pdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        dz = dz * (_phi(z) + z * pdf)
    got = {"dx": torch.mm(dz, s["W"].double()),
           "dW": torch.mm(dz.t().contiguous(), s["x"].double())}
    if s["bias"]:
        got["db"] = dz.sum(dim=0)
    return got


def _exact_norm(s):
    h = s["x"].double()
    if s["r"] is not None:
        h = (h + s["r"].double()).to(s["x"].dtype).double()   # the stream as it is kept
    var, mean = torch.var_mean(h, dim=1, correction=0)
    rstd = (var + EPS).rsqrt()
    y = (h - mean[:, None]) * rstd[:, None] * s["w"].double()
    if s["b"] is not None:
        y = y + s["b"].double()
    got = {"out": y, "mean": mean, "rstd": rstd}
    if s["r"] is not None:
        got["h"] = h
    return got


def _exact_norm_bwd(s):
    x, dy, w = s["x"].double(), s["dout"].double(), s["w"].double()
    mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    d = x.shape[1]
    xh = (x - mean) * rstd
    a = (dy * w).sum(dim=1, keepdim=True) / d
    c = (dy * w * xh).sum(dim=1, keepdim=True) / d
    dx = (dy * w - a - c * xh) * rstd
    if s["r"] is not None:
        dx = dx + s["r"].double()
    got = {"dx": dx, "dw": (dy * xh).sum(dim=0)}
    if s["bias"]:
        got["db"] = dy.sum(dim=0)
    return got


def exact(case, seed):
    s = _inputs(case, seed)
    return {"few": _exact_few, "linear": _exact_linear, "linear_bwd": _exact_linear_bwd,
            "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}[case["op"]](s)
