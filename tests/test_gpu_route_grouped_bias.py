"""The router with groups under large selection biases: which groups stay is decided as
in 64 bits, whatever the biases of a group's two largest values cancel or add up to.

References in 64 bits round v = s + bias to half a unit of the bias (2^-53 B), a sum of
two such values to 2^-52 B, and so does the kernel's own 64-bit form: two groups are in a
certain order where their sums differ by more than 2^-50 B + 2^-48 (the second term: the
scores' own roundings).  Only those tokens are compared."""
import pytest
import torch

import gate_ref as G
from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu


def group_sums(ref, bias, groups):
    v = ref["s"] + bias.cpu().double()
    return v.view(v.shape[0], groups, -1).topk(2, dim=2).values.sum(2)


def check(z, k, bias, groups, keep, score, size):
    """Tokens in a certain order take the reference's experts; returns how many there are."""
    r = ops.moe_route_grouped(z, k, score=score, bias=bias, groups=groups, keep_groups=keep, group_score="top2")
    ref = G.route(z, k, sigmoid=score == "sigmoid", bias=bias, groups=groups, keep=keep, top2=True)
    value = group_sums(ref, bias, groups).sort(1, descending=True).values
    certain = value[:, keep - 1] - value[:, keep] > 2.0 ** -50 * size + 2.0 ** -48
    assert torch.equal(r.experts.cpu().long()[certain], ref["experts"][certain])
    return int(certain.sum())


@pytest.mark.parametrize("size", [2.0, 64.0, 1024.0, 2.0 ** 20])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_biases_that_cancel_in_a_group(size, score):
    """One group has biases +size and -size, the other none: the sums of scores differ by
    up to the fp32 rounding of a value of that size, and some steps more."""
    T = 4000
    g = torch.Generator().manual_seed(int(size))
    z = torch.randn(T, 4, generator=g)
    z[:, 2] = z[:, 0] + (2 * torch.rand(T, generator=g) - 1) * min(size * 2.0 ** -20, 0.5)
    z[:, 3] = z[:, 1]
    bias = torch.tensor([size, -size, 0.0, 0.0], device="cuda")
    assert check(z.cuda(), 2, bias, 2, 1, score, size) > T // 2


@pytest.mark.parametrize("E,groups,keep,k", [(64, 8, 4, 6), (256, 8, 3, 8), (384, 6, 2, 8), (1020, 17, 6, 8)])
@pytest.mark.parametrize("size", [1024.0, 2.0 ** 20])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_every_group_cancels(E, groups, keep, k, size, score):
    """A positive bias for one expert of each group, the negative one for the others:
    every group's value is the sum of two scores."""
    T = 300
    g = torch.Generator().manual_seed(E)
    z = torch.randn(T, E, generator=g).cuda()
    bias = torch.full((groups, E // groups), -size)
    bias[:, 1] = size
    assert check(z, k, bias.reshape(-1).cuda(), groups, keep, score, size) > T // 2


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_sums_past_the_range_of_fp32(score, sign):
    """Two biases whose sum is no fp32 number: the groups keep their order."""
    T = 70
    z = torch.randn(T, 8, generator=torch.Generator().manual_seed(1)).cuda()
    bias = sign * torch.tensor([3e38, 2e38, 2.9e38, 2.5e38, 2.8e38, 3.1e38, 2.7e38, 1e38], device="cuda")
    assert check(z, 4, bias, 4, 2, score, 3.1e38) == T
