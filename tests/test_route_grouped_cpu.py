"""Refusals of the grouped router's entry points (host validation; nothing is
launched) and its reference's own pins."""
import pytest
import torch

import gate_ref as G
from fp8_block_scaled_x128_amd import ops

P = 1 << 20                                   # never dereferenced: validation fails first
NULL, SHAPE, STRIDE, ALIGN, UNSUPPORTED = 1, 2, 3, 4, 5


def route(z=P, T=8, E=16, ld=16, type_=1, k=2, score=1, bias=None, groups=4, keep=2, gs=1, renorm=1, scale=1.0, mask=None,
          experts=P, weights=P, counts=P, offsets=P, row_token=P, token_rows=P, total=P, loss=P, ws=None, wsn=0):
    return ops.fp8_moe_route_grouped(z, T, E, ld, type_, k, score, bias, groups, keep, gs, renorm, scale, mask, experts,
                                     weights, counts, offsets, row_token, token_rows, total, loss, ws, wsn, stream=0,
                                     raise_on_error=False)


@pytest.mark.parametrize("want,a", [
    (SHAPE, dict(T=-1)), (SHAPE, dict(T=(1 << 22) + 1)), (SHAPE, dict(E=0)), (SHAPE, dict(E=1025)), (SHAPE, dict(k=0)),
    (SHAPE, dict(k=17)), (SHAPE, dict(groups=0)), (SHAPE, dict(groups=3)), (SHAPE, dict(E=650, ld=650, groups=65)),
    (SHAPE, dict(keep=0)), (SHAPE, dict(keep=5)), (SHAPE, dict(keep=1, k=5)), (STRIDE, dict(ld=15)),
    (UNSUPPORTED, dict(type_=2)), (UNSUPPORTED, dict(score=2)), (UNSUPPORTED, dict(gs=2)), (UNSUPPORTED, dict(renorm=2)),
    (UNSUPPORTED, dict(scale=float("inf"))), (UNSUPPORTED, dict(scale=float("nan"))), (NULL, dict(z=None)),
    (NULL, dict(experts=None)), (NULL, dict(weights=None)), (NULL, dict(counts=None)), (NULL, dict(offsets=None)),
    (NULL, dict(row_token=None)), (NULL, dict(token_rows=None)), (NULL, dict(total=None)), (NULL, dict(loss=None)),
    (NULL, dict(T=100)), (SHAPE, dict(T=100, ws=P, wsn=64)), (ALIGN, dict(T=100, ws=P + 8, wsn=1 << 20)),
    (ALIGN, dict(bias=P + 2)), (ALIGN, dict(z=P + 2))])
def test_route_refuses(want, a):
    assert route(**a) == want


def back(z=P, T=8, E=16, ld=16, type_=1, k=2, score=1, renorm=1, scale=1.0, experts=P, counts=P, total=P, dw=P, dl=P, out=P,
         ldd=16):
    return ops.fp8_moe_route_grouped_backward(z, T, E, ld, type_, k, score, renorm, scale, experts, counts, total, dw, dl,
                                              out, ldd, stream=0, raise_on_error=False)


@pytest.mark.parametrize("want,a", [
    (SHAPE, dict(E=0)), (UNSUPPORTED, dict(score=-1)), (UNSUPPORTED, dict(scale=float("nan"))), (NULL, dict(z=None)),
    (NULL, dict(total=None)), (NULL, dict(out=None)), (NULL, dict(dw=None, dl=None)), (NULL, dict(experts=None)),
    (NULL, dict(counts=None)), (STRIDE, dict(ldd=15)), (ALIGN, dict(total=P + 1)), (ALIGN, dict(dw=P + 2))])
def test_backward_refuses(want, a):
    assert back(**a) == want


def test_bias_update_refuses_and_empty_calls():
    f = lambda b=P, c=P, E=8, r=0.1: ops.fp8_moe_bias_update(b, c, E, r, stream=0, raise_on_error=False)
    assert f(E=0) == SHAPE and f(E=1025) == SHAPE and f(b=None) == NULL and f(c=None) == NULL
    assert f(r=float("inf")) == UNSUPPORTED and f(b=P + 2) == ALIGN
    assert back(T=0) == 0


def test_reference_selection():
    """Hand-made tokens: groups by sum and by largest value, ties, a bias that
    changes the selection and not the weights."""
    z = torch.tensor([[3.0, -3.0, 1.0, 1.0, 0.0, 0.0]])
    top2 = G.route(z, 2, sigmoid=True, groups=3, keep=1, top2=True)
    most = G.route(z, 2, sigmoid=True, groups=3, keep=1, top2=False)
    assert top2["experts"].tolist() == [[2, 3]] and most["experts"].tolist() == [[0, 1]]
    bias = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.9, 0.0])
    b = G.route(z, 2, sigmoid=True, bias=bias)
    assert b["experts"].tolist() == [[4, 0]]
    s = torch.sigmoid(torch.tensor([0.0, 3.0], dtype=torch.float64))
    assert torch.allclose(b["weights"][0], s / s.sum(), rtol=1e-12)
    assert G.route(torch.zeros(1, 6), 3, sigmoid=False, groups=3, keep=2)["experts"].tolist() == [[0, 1, 2]]


def test_reference_gradient_against_autograd():
    z = torch.randn(7, 12, generator=torch.Generator().manual_seed(2)).double()
    dw, dl = torch.randn(7, 3).double(), torch.tensor([0.3, 0.2]).double()
    for sigmoid in (True, False):
        for renorm in (True, False):
            ref = G.route(z, 3, sigmoid=sigmoid, groups=4, keep=2, renorm=renorm, scale=1.5)
            x = z.clone().requires_grad_(True)
            want, = torch.autograd.grad(G.objective(ref, x, dw, dl, sigmoid=sigmoid, renorm=renorm, scale=1.5), x)
            got, mag = G.grad(ref, dw, dl, sigmoid=sigmoid, renorm=renorm, scale=1.5)
            assert ((got - want).abs() <= 1e-12 * mag + 1e-15).all()
