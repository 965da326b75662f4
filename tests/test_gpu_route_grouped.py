"""The router with scores, a selection bias and groups, its gradient and the bias
update against 64-bit references; whole numbers must be equal.

Bounds in roundings of U = 2^-24: a sigmoid's exponential costs (2 |z| + 2) U, its
reciprocal, sum and product 4; an exponential of an fp32 difference (2 |d| + 4) U; a
token's sum is a chain of at most 32 terms per lane and 6 lane steps.  The
probability sums add a chain over a workgroup's tokens (64), its 16 waves and the
workgroups (T / 64)."""
import pytest
import torch

import block_ref as R
import gate_ref as G
from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WHOLE = ("experts", "counts", "offsets", "row_token", "token_rows")
U = R.U


def logits_of(T, E, dt, seed, disabled=0, pad=0, steps=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E + pad, generator=g) + 0.7 * torch.randn(E + pad, generator=g)
    if steps:
        z = torch.round(z * steps) / steps
    z = z.to(dt)
    if disabled:
        z[:, torch.randperm(E, generator=g)[:disabled]] = -torch.inf
    return z.cuda()[:, :E]


def bias_of(E, seed, size=0.1):
    return (size * torch.randn(E, generator=torch.Generator().manual_seed(seed + 99))).cuda()


def size(ref):
    """max |z| (sigmoid) and max |z - m| of each token, over finite logits."""
    z = torch.where(torch.isfinite(ref["z"]), ref["z"], torch.zeros_like(ref["z"]))
    return z.abs().amax(1) * 2


def check(z, k, r, *, sigmoid, renorm=True, **o):
    ref = G.route(z, k, sigmoid=sigmoid, renorm=renorm, **o)
    for n in WHOLE:
        assert torch.equal(getattr(r, n).cpu().long(), ref[n].long()), n
    big = size(ref)
    c = (4 * big + 160 + k)[:, None]
    err = (R.d(r.weights) - ref["weights"]).abs()
    assert (err <= 2 * c * U * ref["weights"].abs() + 1e-37).all(), "weights"
    live = ref["live"]
    assert torch.equal(R.d(r.lse)[~live], ref["total"][~live])
    el = (R.d(r.lse) - ref["total"])[live].abs()
    lim = (4 * big + 60)[live] * U * (ref["total"].abs()[live] if sigmoid else 1 + ref["total"].abs()[live])
    assert (el <= lim + 1e-37).all(), "total"
    cl = 220 + z.shape[0] / 64 + 4 * float(big.max()) if z.shape[0] else 0
    assert abs(float(r.loss[0]) - float(ref["loss"][0])) <= cl * U * float(ref["loss"][0]), "balance"
    if sigmoid:
        assert float(r.loss[1]) == 0
    else:
        t = ref["total"][live].abs()
        slack = float((2 * t * (4 * big[live] + 60) * U * (1 + t)).sum()) / ref["n"]
        assert abs(float(r.loss[1]) - float(ref["loss"][1])) <= slack + cl * U * float(ref["loss"][1]) + 1e-37, "z loss"
    return ref


def check_grad(z, k, r, ref, *, score, renorm, scale, dw, dl):
    out = ops.moe_route_grouped_backward(z, r.experts, r.counts, r.lse, dweights=dw, dloss=dl, score=score,
                                         renorm=renorm, scale=scale)
    want, mag = G.grad(ref, dw, dl, sigmoid=score == "sigmoid", renorm=renorm, scale=scale)
    R.close(out, want, mag, (16 * size(ref) + 400 + 2 * k)[:, None], "dlogits")
    return out


CASES = [(8, 1, 1, 1), (16, 4, 2, 8), (24, 6, 3, 4), (60, 4, 2, 4), (64, 8, 4, 6), (64, 64, 5, 5), (96, 3, 2, 32),
         (128, 8, 4, 8), (130, 2, 1, 7), (256, 8, 4, 8), (256, 1, 1, 8), (260, 13, 5, 8), (384, 6, 4, 8), (495, 33, 9, 8),
         (512, 16, 5, 8), (720, 9, 4, 6), (1023, 3, 2, 20), (1024, 32, 8, 8), (1020, 17, 6, 8)]


@pytest.mark.parametrize("E,groups,keep,k", CASES)
@pytest.mark.parametrize("T", [1, 65, 200])
@pytest.mark.parametrize("dt,score,top2,renorm,scale", [(F32, "sigmoid", True, True, 2.5), (BF, "softmax", False, False, 1.0),
                                                         (F32, "softmax", True, True, 1.0), (BF, "sigmoid", False, True, 0.7)])
def test_route_and_gradient(T, E, groups, keep, k, dt, score, top2, renorm, scale):
    z = logits_of(T, E, dt, T + E, pad=T % 3)
    g = torch.Generator().manual_seed(T)
    dw, dl = torch.randn(T, k, generator=g).cuda(), torch.tensor([0.3, 0.2], device="cuda")
    for bias in (None, bias_of(E, E, 0.1 if score == "sigmoid" else 4.0 / E)):
        r = ops.moe_route_grouped(z, k, score=score, bias=bias, groups=groups, keep_groups=keep,
                                  group_score="top2" if top2 else "max", renorm=renorm, scale=scale)
        ref = check(z, k, r, sigmoid=score == "sigmoid", bias=bias, groups=groups, keep=keep, top2=top2, renorm=renorm,
                    scale=scale)
        for a, b in ((dw, dl), (dw, None), (None, dl)):
            check_grad(z, k, r, ref, score=score, renorm=renorm, scale=scale, dw=a, dl=b)


@pytest.mark.parametrize("E,groups,keep,k", [(32, 4, 2, 4), (128, 8, 4, 8), (256, 8, 3, 8), (1024, 16, 4, 8)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_values_closer_than_fp32(E, groups, keep, k, score):
    """Scores a few 1e-9 apart (fp32 rounds them together) and equal ones, under one
    bias: the order is that of 64 bits, ties go to the lower expert or group."""
    T = 150
    g = torch.Generator().manual_seed(E)
    z = (torch.randint(0, 40, (T, E), generator=g) * 4e-9).float().cuda()
    bias = torch.full((E,), 0.25, device="cuda")
    for b in (bias, None):
        for top2 in (True, False):
            r = ops.moe_route_grouped(z, k, score=score, bias=b, groups=groups, keep_groups=keep,
                                      group_score="top2" if top2 else "max")
            ref = G.route(z, k, sigmoid=score == "sigmoid", bias=b, groups=groups, keep=keep, top2=top2)
            decided = torch.ones(T, dtype=torch.bool)
            if top2:
                # z = 4e-9 i, i < 40: pairs of equal i + j have sums that differ only
                # by the score's curvature, below (1.6e-7)^2 = 2.6e-14 of s, or 8e-16
                # with s = 1 / 32 (softmax) and less for the sigmoid, whose curvature
                # at 0 is 0: a few roundings of 64 bits, which do not order them.
                # Tokens whose cut lies there are left out.
                v = ref["s"] if b is None else ref["s"] + 0.25
                value = v.view(T, groups, E // groups).topk(2, dim=2).values.sum(2).sort(1, descending=True).values
                decided = value[:, keep - 1] - value[:, keep] > 2.0 ** -50
                assert decided.any()      # of 1024 experts most groups hold the two largest logits
            assert torch.equal(r.experts.cpu().long()[decided], ref["experts"][decided]), (top2, b is None)
            if decided.all():
                for n in WHOLE:
                    assert torch.equal(getattr(r, n).cpu().long(), ref[n].long()), (n, top2, b is None)


@pytest.mark.parametrize("T", [5, 64, 200, 777])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masks_and_disabled_experts(T, dt, score):
    """Masked tokens (anything in their logits), experts disabled by logit or bias,
    groups without experts, tokens with fewer than k experts or none, equal logits."""
    E, k, groups, keep = 24, 4, 6, 2
    z = logits_of(T, E, dt, T, steps=2).clone()
    bias = bias_of(E, 3)
    bias[7] = -torch.inf
    z[:, 8:12] = -torch.inf                     # a whole group
    z[:, 20] = -torch.inf
    mask = torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7
    z[~mask.cuda()] = torch.nan
    z[0] = -torch.inf
    z[1, 2:] = -torch.inf
    z[2] = torch.finfo(dt).min
    z[3] = 0.0
    z[3, ::2] = -0.0
    mask[:4] = True
    mask = mask.cuda()
    for b in (bias, None):
        for top2 in (True, False):
            o = dict(bias=b, groups=groups, renorm=True, mask=mask)
            r = ops.moe_route_grouped(z, k, score=score, keep_groups=keep, group_score="top2" if top2 else "max", **o)
            ref = G.route(z, k, sigmoid=score == "sigmoid", keep=keep, top2=top2, **o)
            for n in WHOLE:
                assert torch.equal(getattr(r, n).cpu().long(), ref[n].long()), n
            assert not ref["live"][0] and int((ref["experts"][1] >= 0).sum()) <= 2
            assert (r.weights[r.experts < 0] == 0).all() and torch.isfinite(r.weights).all()
            dw = torch.randn(T, k, device="cuda")
            dw[r.experts < 0] = torch.nan          # slots without an expert are not read
            dl = torch.tensor([0.3, 0.0], device="cuda")
            out = ops.moe_route_grouped_backward(z, r.experts, r.counts, r.lse, dweights=dw, dloss=dl, score=score)
            want, mag = G.grad(ref, dw, dl, sigmoid=score == "sigmoid", renorm=True, scale=1.0)
            c = torch.where(size(ref) < 100, 16 * size(ref) + 400, torch.full_like(size(ref), 500.0))[:, None]
            R.close(out, want, mag, c, "dlogits")
            assert (out[~mask] == 0).all() and (out[0] == 0).all()


def test_none_masked_and_not_a_number():
    z = logits_of(100, 16, F32, 1).clone()
    for score in ("sigmoid", "softmax"):
        o = dict(score=score, groups=4, keep_groups=2, bias=bias_of(16, 1))
        r = ops.moe_route_grouped(z, 2, mask=torch.zeros(100, dtype=torch.bool, device="cuda"), **o)
        assert (r.experts == -1).all() and (r.counts == 0).all() and (r.offsets == 0).all() and (r.loss == 0).all()
        assert (r.token_rows == -1).all() and (r.row_token == 0).all() and (r.weights == 0).all()
        r = ops.moe_route_grouped(z[:0], 2, **o)
        assert (r.counts == 0).all() and (r.offsets == 0).all() and (r.loss == 0).all()
        y = z.clone()
        y[7, 3] = torch.nan
        r = ops.moe_route_grouped(y, 2, **o)
        assert int(r.experts[7, 0]) == (3 if score == "sigmoid" else int(r.experts[7, 0]))
        assert torch.isnan(r.weights[7]).any() and torch.isnan(r.loss[0])
        ok = [i for i in range(100) if i != 7]
        assert torch.isfinite(r.weights[ok]).all() and torch.isfinite(r.lse[ok]).all()
    # every logit of a sigmoid far down: scores of 0, and no division by it
    r = ops.moe_route_grouped(torch.full((3, 16), -200.0, device="cuda"), 2)
    assert (r.weights == 0).all() and r.experts.tolist() == [[0, 1]] * 3 and (r.lse == 0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the 64-bit scalar with the selection and counts held:
    step 1e-5, second-order error below 1e-8 of the terms."""
    T, E, k, scale = 12, 20, 3, 1.7
    z = logits_of(T, E, F32, 3)
    o = dict(groups=4, renorm=renorm, scale=scale, bias=bias_of(E, 5))
    r = ops.moe_route_grouped(z, k, score=score, keep_groups=2, **o)
    ref = G.route(z, k, sigmoid=score == "sigmoid", keep=2, **o)
    g = torch.Generator().manual_seed(4)
    dw, dl = torch.randn(T, k, generator=g), torch.tensor([0.3, 0.2])
    out = R.d(ops.moe_route_grouped_backward(z, r.experts, r.counts, r.lse, dweights=dw.cuda(), dloss=dl.cuda(),
                                             score=score, renorm=renorm, scale=scale))
    _, mag = G.grad(ref, dw, dl, sigmoid=score == "sigmoid", renorm=renorm, scale=scale)
    f = lambda x: float(G.objective(ref, x, dw.double(), dl.double(), sigmoid=score == "sigmoid", renorm=renorm,
                                    scale=scale))
    for t in range(T):
        for e in range(E):
            h = torch.zeros(T, E, dtype=torch.float64)
            h[t, e] = 1e-5
            diff = (f(ref["z"] + h) - f(ref["z"] - h)) / 2e-5
            assert abs(diff - float(out[t, e])) <= 1e-5 * float(mag[t, e]) + 1e-9


@pytest.mark.parametrize("T,E", [(32769, 64), (40000, 256)])
def test_many_tokens(T, E):
    """Past the workgroups that one launch adds up directly; checked by properties
    and on every 97th token."""
    z, bias = logits_of(T, E, F32, T), bias_of(E, 2)
    o = dict(groups=8, bias=bias)
    r = ops.moe_route_grouped(z, 6, keep_groups=3, **o)
    ref = G.route(z[::97], 6, sigmoid=True, keep=3, **o)
    assert torch.equal(r.experts[::97].cpu().long(), ref["experts"])
    e = r.experts.long()
    assert torch.equal(r.counts[:E].long(), torch.bincount(e.reshape(-1), minlength=E)) and int(r.counts[E]) == T
    order = e.reshape(-1).sort(stable=True).indices
    assert torch.equal(r.row_token.long(), order // 6)
    assert torch.equal(r.token_rows.reshape(-1)[order].long(), torch.arange(T * 6, device="cuda"))


@pytest.mark.parametrize("E", [1, 2, 60, 128, 1000, 1024])
def test_bias_update(E):
    g = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 9, (E + 1,), generator=g, dtype=torch.int32)
    counts[E] = 12345
    if E > 100:
        counts[:E] += 2000000000 // E * 3        # sums past 32 bits
    bias = torch.randn(E, generator=g)
    c = counts[:E].long()
    want = bias + 0.001 * torch.sign((c.sum() - c * E).float())
    b = bias.cuda()
    assert ops.moe_bias_update(b, counts.cuda(), 0.001) is b
    assert torch.equal(b.cpu(), want)
    b = bias.cuda()
    ops.moe_bias_update(b, counts[:E].cuda(), 0.001)
    assert torch.equal(b.cpu(), want)


def test_graph_and_streams():
    """Captured routing and gradient replay with new logits in place; another
    stream's calls with their own workspace run beside them."""
    T, E, k = 3000, 128, 8
    o = dict(groups=8, keep_groups=4, bias=bias_of(E, 1), scale=2.5)
    z, dw = logits_of(T, E, F32, 1).clone(), torch.randn(T, k, device="cuda")
    r = ops.moe_route_grouped(z, k, **o)
    back = lambda z, r, out=None: ops.moe_route_grouped_backward(z, r.experts, r.counts, r.lse, dweights=dw, scale=2.5,
                                                                 out=out)
    d = back(z, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_route_grouped(z, k, out=r, **o)
        back(z, r, d)
        ops.moe_bias_update(o["bias"], r.counts, 0.01)
    other, side = logits_of(T, E, F32, 7), torch.cuda.Stream()
    alone = ops.moe_route_grouped(other, k, **{**o, "bias": None})
    torch.cuda.synchronize()
    for i in range(4):
        z.copy_(logits_of(T, E, F32, 20 + i))
        before = o["bias"].clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            beside = ops.moe_route_grouped(other, k, **{**o, "bias": None})
        graph.replay()
        torch.cuda.synchronize()
        e = ops.moe_route_grouped(z, k, **{**o, "bias": before})
        ed = back(z, e)
        torch.cuda.synchronize()
        for a, b in zip(r[:8], e[:8]):
            assert torch.equal(a, b)
        assert torch.equal(d, ed)
        assert torch.equal(ops.moe_bias_update(before, e.counts, 0.01), o["bias"])
        for a, b in zip(beside[:8], alone[:8]):
            assert torch.equal(a, b)


def test_moe_layer_with_this_router():
    """moe_forward_routed with the grouped router equals the chain of calls; the
    integer layer takes the same maps."""
    T, H, I, E, k = 200, 256, 128, 8, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(BF).cuda()
    wgu = (0.05 * torch.randn(E, 2 * I, H, generator=g)).to(BF).cuda()
    wd = (0.05 * torch.randn(E, I, H, generator=g)).to(BF).cuda()
    qgu, sgu, _ = ops.quant_block2d(wgu)
    _, sdt, qdt = ops.quant_block2d(wd, transposed=True)
    z = logits_of(T, E, F32, 2)
    opt = dict(score="sigmoid", bias=bias_of(E, 1), groups=4, keep_groups=2, scale=2.5)
    codes = ops.quant_rowblock(x)
    out, r, y = ops.moe_forward_routed(codes, z, k, qgu, sgu, qdt, sdt, router=opt)
    alone = ops.moe_route_grouped(z, k, **opt)
    for a, b in zip(r[:8], alone[:8]):
        assert torch.equal(a, b)
    want = ops.moe_forward(x, qgu, sgu, qdt, sdt, r.offsets, r.row_token, r.token_rows, r.weights)
    assert torch.equal(out, want)
    q8, s8 = ops.i8_quant(wgu.view(E * 2 * I, H))
    wdt = wd.transpose(1, 2).contiguous()
    qd8, sd8 = ops.i8_quant(wdt.view(E * H, I))
    got = ops.i8_moe_forward(x, q8.view(E, 2 * I, H), s8.view(E, 2 * I), qd8.view(E, H, I), sd8.view(E, H), r.offsets,
                             r.row_token, r.token_rows, r.weights)
    assert got.shape == out.shape and torch.isfinite(got).all()


def test_refusals_of_the_conveniences():
    z = torch.randn(8, 16, device="cuda")
    for bad in (dict(score="relu"), dict(group_score="mean"), dict(bias=torch.zeros(15, device="cuda")),
                dict(bias=torch.zeros(16, device="cuda", dtype=BF)), dict(mask=torch.ones(7, dtype=torch.bool, device="cuda"))):
        with pytest.raises(ValueError):
            ops.moe_route_grouped(z, 2, **bad)
    for bad in (dict(groups=3), dict(groups=4, keep_groups=5), dict(groups=8, keep_groups=1, top_k=3), dict(scale=float("nan"))):
        with pytest.raises(ops.Fp8bsError):
            ops.moe_route_grouped(z, **{"top_k": 2, **bad})
    with pytest.raises(ValueError):
        ops.moe_bias_update(torch.zeros(4, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda"), 0.1)
