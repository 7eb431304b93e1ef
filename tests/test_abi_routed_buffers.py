"""The layer for a given routing on the host: a misaligned routing, and a written
buffer that shares bytes with the routing, with another one or (dgate) with an input,
are refused before anything is enqueued (the pointers are never dereferenced)."""
import ctypes

import pytest

from sparse_mixture_experts_20_amd import binding as B
from tests.test_abi_block import ALIGN, ARG, BF16, F32, UNSUP, WS, t

P = 1 << 34     # apart from each other by more than any buffer here
N, D, E, FF, K = 40, 64, 4, 128, 2
NAMES = ("x", "wu", "wd", "out", "ws", "idx", "gate", "slot", "used", "demand", "drops", "sum",
         "dout", "dx", "dg", "dwu", "dwd", "bu", "bd", "dbu", "dbd")
OWN = {n: (i + 1) * P for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def L():
    return B.lib()


def _size(L, name, back):
    return dict(x=2 * N * D, out=2 * N * D, dout=2 * N * D, idx=4 * N * K, gate=4 * N * K,
                slot=4 * N * K, used=4 * E, demand=4 * E, drops=4 * E, sum=4 * E, dx=4 * N * D,
                dg=4 * N * K, wu=2 * E * FF * D, wd=2 * E * FF * D, dwu=4 * E * FF * D,
                dwd=4 * E * FF * D, bu=4 * E * FF, bd=4 * E * D, dbu=4 * E * FF, dbd=4 * E * D,
                ws=(L.moe_backward_workspace_size if back else L.moe_workspace_size)(
                    N, D, E, FF, K, 1.0, BF16))[name]


def _call(L, back, p):
    st = B.MoeStats(None, p["ws"], 1 << 40, p["idx"], p["gate"], p["slot"], p["used"], -1,
                    p["demand"], p["drops"], p["sum"], None)
    bu, bd = t(F32, E, FF, ptr=p["bu"]), t(F32, E, D, ptr=p["bd"])
    at = [ctypes.cast(ctypes.c_char_p(b), ctypes.c_void_p) for b in (bu, bd)]
    o = ctypes.byref(B.MoeExpertOpts(B.MOE_ACT_GELU, *at, 0.0, 0, 0))
    x = t(BF16, N, D, ptr=p["x"])
    wu, wd = t(BF16, E, FF, D, ptr=p["wu"]), t(BF16, E, D, FF, ptr=p["wd"])
    if back:
        rc = L.moe_backward_routed(
            x, wu, wd, o, K, 1.0, t(BF16, N, D, ptr=p["dout"]), t(F32, N, D, ptr=p["dx"]),
            t(F32, N, K, ptr=p["dg"]), t(F32, E, FF, D, ptr=p["dwu"]),
            t(F32, E, D, FF, ptr=p["dwd"]), t(F32, E, FF, ptr=p["dbu"]),
            t(F32, E, D, ptr=p["dbd"]), ctypes.byref(st))
    else:
        rc = L.moe_forward_routed(x, wu, wd, o, K, 1.0, t(BF16, N, D, ptr=p["out"]),
                                  ctypes.byref(st))
    assert st.capacity == -1      # refused before anything was written
    return rc


@pytest.mark.parametrize("back", [False, True])
def test_misaligned_routing(L, back):
    for name in ("idx", "gate"):
        for off in (1, 2, 3):
            assert _call(L, back, {**OWN, name: OWN[name] + off}) == ALIGN, name


WRITTEN = {False: ("out", "ws", "slot", "used", "demand", "drops", "sum"),
           True: ("dx", "dg", "dwu", "dwd", "dbu", "dbd", "ws", "slot", "used", "demand",
                  "drops", "sum")}


def _pairs(back):
    for a in WRITTEN[back]:
        for b in ("idx", "gate", *WRITTEN[back]):
            if a != b:
                yield a, b
        if a == "dg":
            yield from ((a, b) for b in ("x", "dout", "wu", "wd", "bu", "bd"))


@pytest.mark.parametrize("back", [False, True])
def test_overlaps(L, back):
    for a, b in _pairs(back):
        n, m = _size(L, b, back), _size(L, a, back)
        first = 256 if a == "ws" else 16     # (kept aligned, so that the overlap is the fault)
        last = OWN[b] + (n - 1) // first * first
        starts = {OWN[b], last}
        if m > first:
            starts.add(OWN[b] - (m - 1) // first * first)
        for where in starts:
            assert _call(L, back, {**OWN, a: where}) == ARG, (a, b, where - OWN[b])


def test_routing_limits(L):
    """Widths past MOE_ROUTE_MAX_WIDTH and, for the backward, rows past
    MOE_ROUTE_MAX_GRAD_ROWS are refused (a launch could not hold them)."""
    wide, rows = (1 << 25) + 8, (1 << 29) + 1
    P40 = 1 << 44
    a = [(i + 1) * P40 for i in range(8)]

    def back(n, d):
        return L.moe_router_backward(
            t(BF16, n, d, ptr=a[0]), t(F32, 8, d, ptr=a[1]), None, 2, a[2],
            t(F32, n, 8, ptr=a[3]), t(F32, n, 2, ptr=a[4]), None, None, t(F32, n, d, ptr=a[5]),
            t(F32, 8, d, ptr=a[6]), a[7], 1 << 43, None)
    for dt in (F32, BF16):
        assert L.moe_router_ex(t(dt, 4, wide, ptr=a[0]), t(F32, 8, wide, ptr=a[1]), None, None, 2,
                               a[2], a[3], None, a[4], 1 << 43, None) == UNSUP
        assert L.moe_router_ex_workspace_size(4, wide, 256, dt) == 0
        assert L.moe_router_ex_workspace_size(4, 1 << 25, 256, dt) > 0
    assert back(4, wide) == UNSUP and back(rows, 8) == UNSUP
    f = L.moe_router_backward_workspace_size
    assert f(4, wide, 8, 2) == 0 and f(rows, 8, 8, 2) == 0
    assert f(4, 1 << 25, 8, 2) > 0 and f(1 << 29, 8, 8, 2) > 0


def test_gates_of_the_backward(L):
    """A misaligned array of gates, or a written buffer over it, where they are read (with
    renormalised gates); elsewhere they are not looked at."""
    a = [(i + 1) * P for i in range(10)]

    def back(gates, renorm=1, **kw):
        o = B.MoeRouterOpts(0, None, 0, 0, 0, renorm, 0.0, gates)
        w = dict(dx=a[6], dW=a[7], ws=a[8], wn=1 << 33)
        w.update(kw)
        return L.moe_router_backward(
            t(BF16, N, D, ptr=a[0]), t(F32, E, D, ptr=a[1]), ctypes.byref(o), K, a[2],
            t(F32, N, E, ptr=a[3]), t(F32, N, K, ptr=a[4]), None, None,
            t(F32, N, D, ptr=w["dx"]), t(F32, E, D, ptr=w["dW"]), w["ws"], w["wn"], None)
    for off in (1, 2, 3):
        assert back(a[5] + off) == ALIGN
        assert back(a[5] + off, renorm=0, wn=16) == WS     # (the next check)
    for name in ("dx", "dW", "ws"):
        assert back(a[5], **{name: a[5]}) == ARG
        assert back(a[5] + 4 * N * K - 4, **{name: a[5]}) == ARG


def test_extents_whose_product_passes_64_bits(L):
    """More weights than a conversion takes (2^35), also where E M K wraps to 0 or below."""
    for E, M, K in ((256, 1 << 28, 1 << 28), (256, 1 << 28, 1 << 27), (1, 1 << 20, 1 << 15),
                    (256, 1 << 14, 1 << 14)):
        q = B.MoeQ4(P, 2 * P, None, 32, 3, (ctypes.c_int64 * 3)(E, M, K))
        W = t(F32, E, M, K, ptr=1 << 50)
        assert L.moe_quantize(W, ctypes.byref(q), None) == UNSUP, (E, M, K)
        assert L.moe_dequantize(ctypes.byref(q), W, None) == UNSUP, (E, M, K)


def test_rows_whose_assignments_pass_64_bits(L):
    """N k that wraps to a small number is no small batch."""
    n = 1 << 62
    a = [(i + 1) << 50 for i in range(8)]
    st = B.MoeStats(None, a[4], 1 << 62, a[2], a[3], None, None, -1)
    for dt in (F32, BF16):
        x, W = t(dt, n, 16, ptr=a[0]), t(F32, 8, 16, ptr=a[1])
        assert L.moe_router_ex(x, W, None, None, 4, a[2], a[3], None, a[4], 1 << 62, None) == UNSUP
        up = t(dt, 8, 32, 16, ptr=a[5])
        assert L.moe_forward_routed(x, up, t(dt, 8, 16, 32, ptr=a[6]), None, 4, 1.0,
                                    t(dt, n, 16, ptr=a[7]), ctypes.byref(st)) == UNSUP
    assert L.moe_router_backward(t(BF16, n, 16, ptr=a[0]), t(F32, 8, 16, ptr=a[1]), None, 4, a[2],
                                 t(F32, n, 8, ptr=a[3]), t(F32, n, 4, ptr=a[4]), None, None, None,
                                 t(F32, 8, 16, ptr=a[5]), a[6], 1 << 62, None) == UNSUP
    assert L.moe_router_backward_workspace_size(n, 16, 8, 4) == 0
    assert L.moe_workspace_size(n, 16, 8, 32, 4, 1.0, BF16) == 0
