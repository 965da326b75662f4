"""The router's gradient beyond one pass of its token loop, against the 64-bit
reference.

The kernel starts 2048 workgroups at most, each with 16 tokens at a time (16
lanes a token, up to 256 experts) or 4 (64 lanes); a group of lanes uses its
LDS row again for its next token.  Tokens of the second and later passes, dead
ones after live ones among them and the other way round, are compared like the
first.

Bounds, in roundings of U = 2^-24 on the terms' magnitude: exp of a difference
d costs 2 |d| + 4; a token's sums are chains of at most 16 terms a lane and 6
lane steps, twice (the probabilities' and the one with f), 44; the products
around them fewer than 40.  A weight is such an exp over a sum of k of them: the
same in |d|, and 2 k with the sum of its gradients."""
import pytest
import torch

import block_ref as R
from fp8_block_scaled_x128_amd import ops
from test_gpu_route import check, logits_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def at_once(E):
    return 2048 * (16 if E <= 256 else 4)


@pytest.mark.parametrize("T,E,k", [(70001, 16, 2), (33000, 60, 4), (33001, 128, 8), (32769, 200, 6), (8300, 300, 4),
                                   (17000, 512, 10), (9001, 1000, 3), (8193, 1024, 32)])
@pytest.mark.parametrize("dt,renorm", [(F32, True), (F32, False), (BF, True)])
def test_gradient_beyond_one_pass(T, E, k, dt, renorm):
    step = at_once(E)
    assert T > step
    z = logits_of(T, E, dt, T + E, disabled=min(3, E - k)).clone()
    g = torch.Generator().manual_seed(T)
    mask = torch.rand(T, generator=g) < 0.8
    mask[step:] = ~mask[:T - step]                  # dead after live, live after dead, in the same lanes
    mask[T - 5:] = False
    z[~mask.cuda()] = torch.nan
    mask = mask.cuda()
    r = ops.moe_route(z, k, renorm=renorm, mask=mask)
    ref = check(z, k, renorm, mask, r)
    dw = torch.randn(T, k, generator=g).cuda()
    dw[r.experts < 0] = torch.nan                   # slots without an expert have no effect
    dl = torch.tensor([0.3 * T, 0.2 * T], device="cuda")        # the losses' part as large as the weights'
    dist = torch.nan_to_num((ref["z"] - ref["lse"][:, None]).abs(), nan=0.0, posinf=0.0)
    for a, b in ((dw, dl), (dw, None), (None, dl)):
        out = ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=a, dloss=b, renorm=renorm)
        want, mag = R.route_grad(ref, k, renorm, a, b)
        R.close(out, want, mag, 96 + 8 * dist + 2 * k, "dlogits")
        assert (out[~mask] == 0).all()


def test_gradient_of_a_token_does_not_depend_on_its_pass():
    """The same token in the first pass and, 32768 tokens on, in the second:
    the same bytes (weights' part only: the losses' depends on the batch)."""
    E, k, step = 100, 6, at_once(100)
    z = logits_of(step, E, F32, 3).contiguous()
    z = torch.cat([z, z[:1000].flip(0)])
    r = ops.moe_route(z, k, renorm=False)
    dw = torch.randn(step, k, generator=torch.Generator().manual_seed(1)).cuda()
    dw = torch.cat([dw, dw[:1000].flip(0)])
    out = ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=dw, renorm=False)
    assert torch.equal(out[step:], out[:1000].flip(0))
