"""A MoE block as a user runs it: the block's input norm with its codes, the
routing from logits, the experts on those codes, the routed combine, the next
norm with the residual add; and the gradients back to the router's logits and
the norm.  Each stage against the calls it orders or a 64-bit reference."""
import numpy as np
import pytest
import torch

import block_ref as R
from fp8_block_scaled_x128_amd import inputs, ops
from gpu_util import dev_bf16

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def layer():
    d = inputs.small_moe(seed=43, tokens=300, hidden=256, experts=8, inter=128, top_k=2)
    qgu, sgu, _ = ops.quant_block2d(dev_bf16(d["w_gu"]))
    wd = dev_bf16(d["w_d"])
    G, I, H = wd.shape
    qdt = torch.empty((G, H, I), dtype=torch.uint8, device="cuda")
    sdt = torch.empty((G, I // 128, H // 128), dtype=F32, device="cuda")
    ops.fp8_quant_block2d(wd, G, I, H, H, None, 0, qdt, I, sdt)
    return d, (qgu, sgu, qdt, sdt)


def test_routing_is_the_host_generators(layer):
    """The device routing of the workload's logits equals the maps that
    inputs.route_topk makes on the host, and moe_forward on either agrees byte
    for byte once the weights are the same."""
    d, weights = layer
    r = d["routing"]
    z = torch.from_numpy(np.ascontiguousarray(d["logits"])).cuda()
    got = ops.moe_route(z, 2)
    assert np.array_equal(got.offsets.cpu().numpy(), r.offsets)
    assert np.array_equal(got.row_token.cpu().numpy(), r.row_token)
    assert np.array_equal(got.token_rows.cpu().numpy(), r.token_rows)
    assert np.array_equal(got.experts.cpu().numpy(), r.topk_experts)
    x = dev_bf16(d["x"])
    a = ops.moe_forward(x, *weights, got.offsets, got.row_token, got.token_rows, got.weights)
    b, rb, _ = ops.moe_forward_routed(ops.quant_rowblock(x), z, 2, *weights)
    assert torch.equal(a, b) and torch.equal(rb.weights, got.weights)


@pytest.mark.parametrize("masked", [False, True])
def test_block_forward_and_backward(layer, masked):
    d, weights = layer
    z = torch.from_numpy(np.ascontiguousarray(d["logits"])).cuda()
    T, H = d["x"].shape
    mask = None
    if masked:
        mask = torch.ones(T, dtype=torch.bool, device="cuda")
        mask[T - 45:] = False
        z = z.clone()
        z[T - 45:] = torch.nan
    g = torch.Generator().manual_seed(2)
    stream = (2 * torch.randn(T, H, generator=g)).cuda()
    w1, w2, w3 = [(1 + 0.1 * torch.randn(H, generator=g)).cuda() for _ in range(3)]
    n1 = ops.block_norm(stream, None, w_pre=w1, h=False)
    out, routing, y = ops.moe_forward_routed((n1.q, n1.s), z, 2, *weights, mask=mask)
    n2 = ops.block_norm(stream, out, w_pre=w2, w_post=w3, scale=0.5)
    h, mh, yr, my = R.norm(stream, out, w2, w3, None, 1, 0.5, 1e-6)
    R.close(n2.h, h, mh, 64, "h")
    R.close(n2.y, yr, my, 64, "y")
    if masked:
        assert (out[T - 45:] == 0).all() and int(routing.counts[-1]) == T - 45
    # the experts see the same codes through the explicit calls
    pos = routing.token_rows.cpu().long()
    yv = torch.where((pos >= 0)[:, :, None], R.d(y)[pos.clamp(min=0)], torch.zeros(1, dtype=torch.float64))
    w = R.d(routing.weights)
    R.close(out, (w[:, :, None] * yv).sum(1), (w[:, :, None] * yv).abs().sum(1), 3, "combine")
    # backward: the next layer's gradients -> block output -> weights -> logits
    dy2, dh2 = torch.randn(T, H, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()
    g2 = ops.block_norm_backward(dy2, dh2, n2.h, out, w_pre=w2, w_post=w3, scale=0.5)
    dyr, dw = ops.moe_combine_backward(g2.dx, y, routing.token_rows, routing.weights)
    dl = torch.tensor([1e-2, 1e-3], device="cuda")
    dz = ops.moe_route_backward(z, routing.experts, routing.weights, routing.counts, routing.lse, dweights=dw, dloss=dl)
    ref = R.norm_grad(dy2, dh2, n2.h, out, w2, w3, None, 1, 0.5, 1e-6)
    R.close(g2.dx, *ref["dx"], 128, "dx")
    want = R.d(g2.dx)[:, None, :] * yv
    R.close(dw, want.sum(2), want.abs().sum(2), H / 64 + 16, "dweights")
    rr = R.route(z, 2, True, mask)
    rr["weights"] = w
    wz, mz = R.route_grad(rr, 2, True, dw, dl)
    dist = torch.nan_to_num(torch.where(mz > 0, (rr["z"] - rr["lse"][:, None]).abs(), torch.zeros_like(mz)), posinf=0.0)
    R.close(dz, wz, mz, 104 + 8 * dist, "dlogits")


def test_no_tokens_and_no_live_tokens(layer):
    """A batch of no tokens, and one whose every token is masked: no expert
    runs, the output is zeros."""
    d, weights = layer
    H = d["x"].shape[1]
    q, s = ops.quant_rowblock(dev_bf16(d["x"]))
    out, r, _ = ops.moe_forward_routed((q[:0], s[:0]), torch.empty(0, 8, device="cuda"), 2, *weights)
    assert out.shape == (0, H) and (r.counts == 0).all()
    z = torch.randn(300, 8, device="cuda")
    out, r, _ = ops.moe_forward_routed((q, s), z, 2, *weights, mask=torch.zeros(300, dtype=torch.bool, device="cuda"))
    assert (out == 0).all() and (r.counts == 0).all()


def test_serving_block_replays_in_a_graph(layer):
    """One decode step's block (norm, routing, routed combine) captured at a
    padded batch and replayed with other masks and logits: the maps stay on
    the device, so one graph serves every batch fill."""
    T, k, H, E = 16, 2, 256, 8
    stream = torch.randn(T, H, device="cuda").to(BF)
    x = torch.randn(T, H, device="cuda").to(BF)
    w = torch.ones(H, dtype=BF, device="cuda")
    z = torch.randn(T, E, device="cuda")
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    y = torch.randn(T * k, H, device="cuda").to(BF)
    out = torch.empty(T, H, dtype=BF, device="cuda")

    def step(o=None, r=None):
        o = ops.block_norm(stream, x, w_pre=w, w_post=w, out=o)
        r = ops.moe_route(z, k, mask=mask, out=r)
        ops.fp8_moe_combine_routed(y, T * k, H, H, r.token_rows, r.weights, T, k, out, H, ops.OUT_BF16)
        return o, r
    o, r = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o, r)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o, r)
    for live in (16, 1, 0, 9):
        z.normal_()
        x.normal_()
        mask.copy_(torch.arange(T, device="cuda") < live)
        for v in (*o, *r[:8], out):
            v.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (*o, *r[:8], out)]
        eo, er = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*eo, *er[:8], out))), live
        assert int(r.counts[-1]) == live


def test_codes_in_a_wider_buffer(layer):
    """Codes whose rows lie in a wider buffer, as the norm writes them through
    `out`, give the same block; codes that do not fit the experts are refused."""
    d, weights = layer
    x = dev_bf16(d["x"])
    T, H = x.shape
    z = torch.from_numpy(np.ascontiguousarray(d["logits"])).cuda()
    w = torch.ones(H, dtype=BF, device="cuda")
    ref = ops.block_norm(x, None, w_pre=w, h=False, y=False)
    wide = torch.full((T, H + 128), 0x55, dtype=torch.uint8, device="cuda")
    n = ops.block_norm(x, None, w_pre=w, h=False, y=False, out=ref._replace(q=wide[:, :H], s=torch.empty_like(ref.s)))
    a, ra, _ = ops.moe_forward_routed((ref.q, ref.s), z, 2, *weights)
    b, rb, _ = ops.moe_forward_routed((n.q, n.s), z, 2, *weights)
    assert torch.equal(a, b) and torch.equal(ra.row_token, rb.row_token)
    for q, s, zz in ((ref.q[:, :128], ref.s[:, :1], z), (ref.q.t().contiguous().t(), ref.s, z),
                     (ref.q, ref.s[:, :1], z), (ref.q, ref.s.double(), z), (ref.q, ref.s, z[:, :4]),
                     (ref.q.cpu(), ref.s, z), (ref.q.view(torch.int8), ref.s, z)):
        with pytest.raises(ValueError):
            ops.moe_forward_routed((q, s), zz, 2, *weights)


def test_whole_block_replays_in_a_graph(layer):
    """Norm, routing, the experts' products, the combine, the next norm and
    the gradients back to the logits in one graph, its temporaries included;
    replayed on new inputs and masks against the eager run."""
    d, weights = layer
    T, H = d["x"].shape
    gen = torch.Generator(device="cuda").manual_seed(4)
    stream, dy, dh = [torch.randn(T, H, device="cuda", generator=gen) for _ in range(3)]
    w = torch.ones(H, device="cuda")
    z = torch.randn(T, 8, device="cuda", generator=gen)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    dl = torch.tensor([1e-2, 1e-3], device="cuda")

    def step():
        n1 = ops.block_norm(stream, None, w_pre=w, h=False, y=False)
        out, r, y = ops.moe_forward_routed((n1.q, n1.s), z, 2, *weights, mask=mask)
        n2 = ops.block_norm(stream, out, w_pre=w, w_post=w)
        g = ops.block_norm_backward(dy, dh, n2.h, out, w_pre=w, w_post=w)
        dyr, dw = ops.moe_combine_backward(g.dx, y, r.token_rows, r.weights)
        dz = ops.moe_route_backward(z, r.experts, r.weights, r.counts, r.lse, dweights=dw, dloss=dl)
        return (*n1[2:], out, *r[:8], *n2, *g[:2], *g[3:5], dw, dz)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for live in (T, 1, 0, 77):
        stream.normal_()
        z.normal_()
        mask.copy_(torch.arange(T, device="cuda") < live)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in held]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), live
