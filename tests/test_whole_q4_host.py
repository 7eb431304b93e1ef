"""The whole-number results that the 4-bit products are compared with, on the CPU: a
mistake planted in them (zeros, a group or the last columns left out, a choice left out,
another zero point, halves of the bytes changed over) changes nearly every element, so
that equality tells it."""
import pytest
import torch

from tests import _plain_q4 as Q, _whole_q4 as H


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _off(a, b):
    return float((a.to(torch.bfloat16) != b.to(torch.bfloat16)).double().mean())


def _swap(w):
    return (w[0] >> 4) | (w[0] << 4)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,K,M,group", [(5, 14336, 64, 64), (3, 160, 33, 32), (33, 1152, 40, 128)])
def test_linear(N, K, M, group, zero):
    s = H.linear_case(_gen(K), N, K, M, group, zero, True, True, device="cpu")
    want = H.linear(s, "none")
    data, sc, zp, W = s["W"]
    # (of a long product one group moves a result by less than a bf16 step now and then)
    least = 0.5 if K > 8192 else 0.8
    bare = s["b"].double() + s["r"].double()
    assert _off(want, bare.expand_as(want)) > least
    for cols in (slice(0, group), slice(K - group, K)):
        V = W.clone()
        V[:, cols] = 0
        assert _off(want, H.linear(dict(s, W=(data, sc, zp, V)), "none")) > least
    other = (torch.full_like(sc, 8.0) if zp is None else zp) + 1
    assert _off(want, H.linear(dict(s, W=(data, sc, other, Q.values(data, sc, other, group))),
                               "none")) > least
    V = Q.values(_swap(s["W"]), sc, zp, group)
    assert _off(want, H.linear(dict(s, W=(data, sc, zp, V)), "none")) > least


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("N,d,E,k,d_ff,group", [(6, 256, 5, 3, 2048, 64), (20, 96, 4, 2, 160, 32)])
def test_experts(N, d, E, k, d_ff, group, zero, odd):
    s = H.experts_case(_gen(d), N, d, E, k, d_ff, group, zero, True, odd, device="cpu")
    want = H.experts(s)
    live = ((s["idx"] >= 0) & (s["idx"] < E))
    rows = live.any(1)
    assert bool((want[~rows] == 0).all()) and bool((~rows).any()) == odd
    assert _off(want[rows], torch.zeros_like(want[rows])) > 0.9
    # one choice left out: every row that has it
    last = torch.where(live, torch.arange(k), -1).amax(1)
    idx = s["idx"].clone()
    idx[rows, last[rows]] = -1
    assert _off(want[rows], H.experts(dict(s, idx=idx))[rows]) > 0.8
    # the gate of one choice doubled
    gate = s["gate"].clone()
    gate[rows, last[rows]] *= 2
    assert _off(want[rows], H.experts(dict(s, gate=gate))[rows]) > 0.8
    # a group of the hidden row left out
    data, sc, zp, W = s["down"]
    V = W.clone()
    V[..., -group:] = 0
    assert _off(want[rows], H.experts(dict(s, down=(data, sc, zp, V)))[rows]) > 0.6


def test_bounds_of_exactness():
    with pytest.raises(AssertionError):
        H.held(torch.tensor([2.0 ** 23]), 0.5)
    assert H.held(torch.tensor([2.0 ** 23 - 1]), 0.5)
