"""The router (fp8_moe_route), its gradient (fp8_moe_route_backward), the
routed combine and the combine's gradient against 64-bit references; whole
numbers must be equal.

Bounds, in roundings of U = 2^-24: exp of an fp32 difference d costs (2 |d| +
4) U; a token's sum is a chain of at most 16 terms per lane and 6 lane steps.
The probability sums add a chain over a workgroup's tokens (64), its 16 waves
and the workgroups (T / 64)."""
import pytest
import torch

import block_ref as R
from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
WHOLE = ("experts", "counts", "offsets", "row_token", "token_rows")


def logits_of(T, E, dt, seed, disabled=0, ties=False, pad=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E + pad, generator=g) + 0.7 * torch.randn(E + pad, generator=g)
    if ties:
        z = torch.round(z)
    z = z.to(dt)
    if disabled:
        z[:, torch.randperm(E, generator=g)[:disabled]] = -torch.inf
    return z.cuda()[:, :E]


def check(z, k, renorm, mask, r):
    T, E = z.shape
    ref = R.route(z, k, renorm, mask)
    for n in WHOLE:
        assert torch.equal(getattr(r, n).cpu().long(), ref[n].long()), n
    used = ref["experts"] >= 0
    top = torch.where(used, ref["z"].gather(1, ref["experts"].clamp(min=0)), torch.zeros_like(ref["weights"]))
    l = torch.where(ref["live"], ref["lse"], torch.zeros_like(ref["lse"]))
    dist = torch.where(used, (top - l[:, None]).abs(), torch.zeros_like(top))
    c = (4 * dist.amax(1, keepdim=True) if T else 0) + 48 + k
    err = (R.d(r.weights) - ref["weights"]).abs()
    assert (err <= c * R.U * ref["weights"] + 1e-37).all(), "weights"
    assert torch.equal(R.d(r.lse)[~ref["live"]], ref["lse"][~ref["live"]])
    el = (R.d(r.lse) - ref["lse"])[ref["live"]].abs()
    # the log of a sum of at most E terms: 40 roundings of the sum, and of the result
    assert (el <= R.U * (40 + 4 * (ref["lse"].abs() + ref["z"].amax(1).abs())[ref["live"]])).all(), "lse"
    cl = 160 + T / 64
    assert abs(float(r.loss[0]) - float(ref["loss"][0])) <= cl * R.U * float(ref["loss"][0]), "balance"
    n = max(1, int(ref["live"].sum()))
    lim = float((2 * l.abs() * (40 + 4 * l.abs() + 4 * torch.where(ref["live"], ref["z"].amax(1), l).abs())).sum()) / n * R.U
    if float(ref["loss"][1]) > torch.finfo(F32).max:      # the square of a logit of fp32's lowest value
        assert float(r.loss[1]) == torch.inf, "z loss"
        return ref
    assert abs(float(r.loss[1]) - float(ref["loss"][1])) <= lim + cl * R.U * float(ref["loss"][1]) + 1e-37, "z loss"
    return ref


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130, 1000])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (16, 16), (17, 3), (60, 4), (64, 6), (128, 8), (129, 8), (256, 8),
                                 (384, 32), (513, 1), (1024, 20)])
@pytest.mark.parametrize("dt,renorm", [(F32, True), (BF, False)])
def test_route_and_gradient(T, E, k, dt, renorm):
    z = logits_of(T, E, dt, T + E, ties=dt == BF, pad=T % 3)
    r = ops.moe_route(z, k, renorm=renorm)
    ref = check(z, k, renorm, None, r)
    g = torch.Generator().manual_seed(T)
    dw, dl = torch.randn(T, k, generator=g).cuda(), torch.tensor([0.3, 0.2], device="cuda")
    for a, b in ((dw, dl), (dw, None), (None, dl)):
        out = ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=a, dloss=b, renorm=renorm)
        want, mag = R.route_grad(ref, k, renorm, a, b)
        dist = (ref["z"] - ref["lse"][:, None]).abs()
        R.close(out, want, mag, 96 + 8 * dist + k, "dlogits")


@pytest.mark.parametrize("T,E,k", [(32768, 16, 2), (32769, 128, 8), (70001, 128, 8), (50000, 300, 4), (40000, 1000, 3)])
def test_many_tokens(T, E, k):
    """Up to and past the workgroups that one launch adds up directly."""
    z = logits_of(T, E, F32, T, disabled=3)
    r = ops.moe_route(z, k)
    check(z, k, True, None, r)


@pytest.mark.parametrize("T", [5, 64, 200, 777])
@pytest.mark.parametrize("dt", [F32, BF])
def test_masks_and_disabled_experts(T, dt):
    """Masked tokens (anything in their logits), disabled experts, tokens with
    fewer than k experts left, tokens with none, equal logits."""
    E, k = 24, 4
    z = logits_of(T, E, dt, T, disabled=5, ties=True).clone()
    mask = torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7
    z[~mask.cuda()] = torch.nan
    z[0] = -torch.inf
    z[1, 2:] = -torch.inf
    z[2] = torch.finfo(dt).min
    z[3] = 0.0
    z[3, ::2] = -0.0
    mask[:4] = True
    mask = mask.cuda()
    r = ops.moe_route(z, k, mask=mask)
    ref = check(z, k, True, mask, r)
    assert not ref["live"][0] and int((ref["experts"][1] >= 0).sum()) <= 2
    assert ref["experts"][3].tolist() == [0, 1, 2, 3]
    assert torch.equal(ops.moe_route(z, k, mask=mask.to(torch.uint8)).token_rows, r.token_rows)
    dw = torch.randn(T, k, device="cuda")
    dw[(r.experts < 0)] = torch.nan            # slots without an expert are not read
    dl = torch.tensor([0.3, 0.2], device="cuda")
    out = ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=dw, dloss=dl)
    want, mag = R.route_grad(ref, k, True, dw, dl)
    dist = torch.where(mag > 0, (ref["z"] - ref["lse"][:, None]).abs(), torch.zeros_like(mag))
    dist = torch.nan_to_num(dist, posinf=0.0)
    R.close(out, want, mag, 96 + 8 * dist + k, "dlogits")
    assert (out[~mask] == 0).all() and (out[0] == 0).all()


def test_all_masked_none_and_not_a_number():
    z = logits_of(100, 16, F32, 1).clone()
    r = ops.moe_route(z, 2, mask=torch.zeros(100, dtype=torch.bool, device="cuda"))
    assert (r.experts == -1).all() and (r.counts == 0).all() and (r.offsets == 0).all() and (r.loss == 0).all()
    assert (r.token_rows == -1).all() and (r.row_token == 0).all() and (r.weights == 0).all()
    r = ops.moe_route(z[:0], 2)
    assert (r.counts == 0).all() and (r.offsets == 0).all() and (r.loss == 0).all()
    # NaN ranks first and shows in its token's weights and in the losses only
    z[7, 3] = torch.nan
    z[9, 4] = torch.inf
    r = ops.moe_route(z, 2)
    ref = R.route(z, 2, True, None)
    for n in WHOLE:
        assert torch.equal(getattr(r, n).cpu().long(), ref[n].long()), n
    assert int(r.experts[7, 0]) == 3 and torch.isnan(r.weights[7]).all() and torch.isnan(r.loss).all()
    ok = [i for i in range(100) if i not in (7, 9)]
    assert torch.isfinite(r.weights[ok]).all() and torch.isfinite(r.lse[ok]).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit scalar with the selection and counts
    held: step 1e-5, second-order error below 1e-8 of the terms."""
    T, E, k = 12, 20, 3
    for renorm in (True, False):
        z = logits_of(T, E, F32, 3)
        r = ops.moe_route(z, k, renorm=renorm)
        dw, dl = torch.randn(T, k, device="cuda"), torch.tensor([0.5, 0.1], device="cuda")
        out = R.d(ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=dw, dloss=dl,
                                         renorm=renorm))
        at, f = r.experts.cpu().long(), R.d(r.counts[:E]) / (T * k)

        def scalar(v):
            p = torch.softmax(v, 1)
            w = p.gather(1, at)
            w = w / w.sum(1, keepdim=True) if renorm else w
            bal = E * (f * p.mean(0)).sum()
            return float((w * R.d(dw)).sum() + R.d(dl)[0] * bal + R.d(dl)[1] * torch.logsumexp(v, 1).square().mean())
        v = torch.randn(T, E, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        diff = (scalar(R.d(z) + 1e-5 * v) - scalar(R.d(z) - 1e-5 * v)) / 2e-5
        terms = float((out * v).abs().sum())
        assert abs(float((out * v).sum()) - diff) <= (256 * R.U + 1e-6) * terms


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 2048), (7, 3, 264), (130, 2, 256), (33, 11, 1000), (40, 32, 64)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_combine_routed_and_gradient(T, k, H, dt):
    """Forward as fp8_moe_combine where every slot has a row; slots without
    one contribute nothing (their y rows hold NaN); the gradient; dy rows that
    no slot names keep their bytes."""
    g = torch.Generator().manual_seed(T * k + H)
    z = torch.randn(T, max(k, 40), generator=g).cuda()
    mask = torch.rand(T, generator=g) < 0.8
    mask[0] = True
    r = ops.moe_route(z, k, mask=mask.cuda())
    rows, n = T * k, int(r.offsets[-1])
    ybuf = torch.full((rows, H + 8), torch.nan, dtype=BF)
    ybuf[:n] = torch.randn(n, H + 8, generator=g).to(BF)
    y = ybuf.cuda()[:, :H]
    out = torch.empty(T, H, device="cuda")
    ops.fp8_moe_combine_routed(y, rows, H, H + 8, r.token_rows, r.weights, T, k, out, H, ops.OUT_FP32)
    pos = r.token_rows.cpu().long()
    yv = torch.where((pos >= 0)[:, :, None], R.d(y)[pos.clamp(min=0)], torch.zeros(1, dtype=torch.float64))
    w = R.d(r.weights)
    R.close(out, (w[:, :, None] * yv).sum(1), (w[:, :, None] * yv).abs().sum(1), k + 1, "combine")
    assert (out[~mask.cuda()] == 0).all()
    if bool(mask.all()):
        same = torch.empty_like(out)
        ops.fp8_moe_combine(y, rows, H, H + 8, r.token_rows, r.weights, T, k, same, H, ops.OUT_FP32)
        assert torch.equal(out, same)
    dout = torch.randn(T, H, generator=g).to(dt).cuda()
    dybuf = torch.full((rows, H + 8), 7.0, dtype=BF, device="cuda")
    dy, dw = ops.moe_combine_backward(dout, y, r.token_rows, r.weights,
                                      out=(dybuf[:, :H], torch.full((T, k), 7.0, device="cuda")))
    want = (R.d(dout)[:, None, :] * yv)
    R.close(dw, want.sum(2), want.abs().sum(2), H / 64 + 16, "dweights")
    v = w[:, :, None] * R.d(dout)[:, None, :]
    live = pos >= 0
    ref = torch.zeros(n, H, dtype=torch.float64)
    ref[pos[live]] = v[live]
    R.close(dy[:n], ref, ref.abs(), 1, "dy")
    assert (dybuf[n:] == 7).all() and (dybuf[:, H:] == 7).all()
    # each output alone
    only = torch.full((T, k), 7.0, device="cuda")
    ops.fp8_moe_combine_backward(dout, H, ops.OUT_FP32 if dt == F32 else ops.OUT_BF16, y, rows, H, H + 8,
                                 r.token_rows, r.weights, T, k, None, 0, only)
    assert torch.equal(only, dw)
    lone = torch.full((rows, H), 7.0, dtype=BF, device="cuda")
    ops.fp8_moe_combine_backward(dout, H, ops.OUT_FP32 if dt == F32 else ops.OUT_BF16, None, rows, H, 0,
                                 r.token_rows, r.weights, T, k, lone, H, None)
    assert torch.equal(lone[:n], dy[:n]) and (lone[n:] == 7).all()


def test_combine_without_rows():
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    out = torch.full((3, 64), 5.0, device="cuda")
    ops.fp8_moe_combine_routed(None, 0, 64, 64, pos, w, 3, 2, out, 64, ops.OUT_FP32)
    assert (out == 0).all()
    dw = torch.full((3, 2), 5.0, device="cuda")
    ops.fp8_moe_combine_backward(out, 64, ops.OUT_FP32, None, 0, 64, 0, pos, w, 3, 2, None, 0, dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("T", [40, 1000, 33000])
def test_route_graph_replays_and_streams(T):
    """Routing and its gradient captured once and replayed on new logits, eager
    calls between; then the same on two streams at once, each with tensors and
    workspace of its own."""
    E, k = 60, 4
    z = logits_of(T, E, F32, 1).contiguous()
    dw, dl = torch.randn(T, k, device="cuda"), torch.tensor([0.3, 0.2], device="cuda")

    def both(z, r=None, o=None):
        r = ops.moe_route(z, k, out=r)
        return r, ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=dw, dloss=dl, out=o)
    r, o = both(z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(z, r, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(z, r, o)
    for rep in range(4):
        z.normal_()
        for v in (*r[:8], o):
            v.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        er, eo = both(z)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*r[:8], o), (*er[:8], eo))), rep
    zs = [logits_of(T, E, F32, s).contiguous() for s in (5, 6)]
    want = [both(v) for v in zs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for rep in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, both(zs[i])))
    torch.cuda.synchronize()
    for i, (er, eo) in got:
        assert all(torch.equal(a, b) for a, b in zip((*er[:8], eo), (*want[i][0][:8], want[i][1])))


def test_refusals():
    z = torch.randn(10, 16, device="cuda")
    with pytest.raises(ValueError):
        ops.moe_route(z.cpu(), 2)
    with pytest.raises(ValueError):
        ops.moe_route(z.half(), 2)
    with pytest.raises(ValueError):
        ops.moe_route(z.t(), 2)
    with pytest.raises(ValueError):
        ops.moe_route(z, 2, mask=torch.ones(9, dtype=torch.bool, device="cuda"))
    with pytest.raises(ops.Fp8bsError):
        ops.moe_route(z, 17)
    with pytest.raises(ops.Fp8bsError):
        ops.moe_route(z[:1].expand(10, 16), 2)
    r = ops.moe_route(z, 2)
    with pytest.raises(ValueError):
        ops.moe_route(z[:9], 2, out=r)
    with pytest.raises(ops.Fp8bsError):
        ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse)
    with pytest.raises(ValueError):
        ops.moe_route_backward(z, r.experts, r.weights, r.counts[:-1], r.lse, dloss=torch.ones(2, device="cuda"))
    y = torch.randn(20, 64, device="cuda").to(BF)
    with pytest.raises(ValueError):
        ops.moe_combine_backward(y[:10], y[:, :56], r.token_rows, r.weights)
    with pytest.raises(ValueError):
        ops.moe_combine_backward(y[:10], y, r.token_rows.long(), r.weights)


def test_rows_past_32_bit_offsets():
    """Logits, their gradient, the experts' rows and the combine's gradient in
    rows 2^30 + 8 elements apart: the last one starts past 2^31 elements."""
    T, E, k, H, ld = 3, 24, 1, 264, 2 ** 30 + 8
    g = torch.Generator().manual_seed(6)
    big = torch.empty(2 * ld + 5 * 512, dtype=BF, device="cuda")
    at = lambda i, c: big[i * 512:i * 512 + 2 * ld + 512].as_strided((T, c), (ld, 1))
    z, y, dout = torch.randn(T, E, generator=g), torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    z, y, dout = [v.to(BF).cuda() for v in (z, y, dout)]
    fz, fy, fdout = at(0, E), at(1, H), at(2, H)
    for far, near in ((fz, z), (fy, y), (fdout, dout)):
        far.copy_(near)
    r, f = ops.moe_route(z, k, renorm=False), ops.moe_route(fz, k, renorm=False)
    assert all(torch.equal(p, q) for p, q in zip(r[:8], f[:8]))
    dy, dw = ops.moe_combine_backward(dout, y, r.token_rows, r.weights)
    fdy, fdw = ops.moe_combine_backward(fdout, fy, f.token_rows, f.weights, out=(at(3, H), torch.empty_like(dw)))
    assert torch.equal(dy, fdy) and torch.equal(dw, fdw)
    a, b = torch.empty(T, H, dtype=BF, device="cuda"), at(4, H)
    ops.fp8_moe_combine_routed(y, T, H, H, r.token_rows, r.weights, T, k, a, H, ops.OUT_BF16)
    ops.fp8_moe_combine_routed(fy, T, H, ld, r.token_rows, r.weights, T, k, b, ld, ops.OUT_BF16)
    assert torch.equal(a, b)
    arg = (r.experts, r.weights, r.counts, r.lse)
    dz = ops.moe_route_backward(z, *arg, dweights=dw, renorm=False)
    fdz = ops.moe_route_backward(fz, *arg, dweights=dw, renorm=False, out=at(3, E))
    assert torch.equal(dz, fdz)


def test_the_largest_router():
    """2^22 tokens, the documented limit: 65536 workgroups' histograms in 256
    runs.  The maps against torch's stable sort, the counts exactly."""
    T, E, k = 2 ** 22, 8, 2
    z = torch.randn(T, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    z = (torch.floor(z * 2.0 ** 16) * 8 + torch.arange(E, device="cuda")) * 2.0 ** -19      # whole multiples: no ties
    r = ops.moe_route(z, k)
    top = torch.topk(z, k, dim=1)
    assert torch.equal(r.experts.long(), top.indices)
    flat = r.experts.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(r.row_token.long(), order // k)
    assert torch.equal(r.token_rows.reshape(-1).long()[order], torch.arange(T * k, device="cuda"))
    counts = torch.stack([(flat == e).sum() for e in range(E)])
    assert torch.equal(r.counts[:E].long(), counts) and int(r.counts[E]) == T
    assert torch.equal(r.offsets[1:].long(), counts.cumsum(0))
    p = torch.softmax(z.double(), 1)
    want = E * float((counts.double() / (T * k) * p.mean(0)).sum())
    # exp 32 and its sum 16; chains over 64 tokens, 16 waves, 256 workgroups,
    # 256 runs and 16 waves again; the product with the counts and its sum 16
    assert abs(float(r.loss[0]) - want) <= (32 + 16 + 64 + 16 + 256 + 256 + 16 + 16) * R.U * want
